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


def test_embed_gradient_of_too_many_rows_is_refused():
    """Its order is quadratic in the rows, and their number of windows has to fit an int."""
    build.build()
    lib = L.load()

    def bwd(n, d_out=F + 1):
        return lib.oomb_embed_bwd(F, n, d_out, 10, 1, 0, 1.0, F, 1, F, 1 << 50, F, None)

    for n in ((1 << 26) + 1, 2 ** 31 - 16, 2 ** 31 - 15, 2 ** 31 - 1):
        assert bwd(n) == 8
    assert bwd(1 << 26) == ALIGN
