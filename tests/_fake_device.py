"""Host tensors that say they are on a device, for tests of what a call checks and passes on (nothing follows them)."""
import torch


class Placed(torch.Tensor):
    """A host tensor whose Python side reports device index ``at``."""
    at = 0

    @staticmethod
    def of(t, at=0):
        p = torch.Tensor._make_subclass(Placed, t)
        p.at = at
        return p

    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.at
