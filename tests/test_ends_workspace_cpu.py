"""Where the calls at a model's two ends ask for a workspace, through the C ABI on the CPU (placeholder pointers; every
call is refused before anything is launched)."""
import paged_sparse_attention_gb300 as L
from paged_sparse_attention_gb300 import build

ALIGN, WORKSPACE = 3, 9
F = 1 << 24  # a placeholder address


def test_layer_norm_backward_asks_only_for_parameter_gradients():
    build.build()
    lib = L.load()

    def bwd(dw, db, n=100, ws=None, size=0, dy=F + 1):  # dy off its element's size: the check behind the workspace's
        return lib.oomb_layer_norm_bwd(F, F, F, F, dy, None, n, 64, 0, F, dw, db, 0, ws, size, None)

    for n in (4, 16, 17, 100):
        assert bwd(None, None, n) == ALIGN
        assert bwd(F, None, n) == WORKSPACE and bwd(None, F, n) == WORKSPACE and bwd(F, F, n) == WORKSPACE
        assert bwd(F, F, n, F, lib.oomb_layer_norm_workspace(n, 64) - 1) == WORKSPACE
        assert bwd(F, F, n, F, lib.oomb_layer_norm_workspace(n, 64)) == ALIGN
