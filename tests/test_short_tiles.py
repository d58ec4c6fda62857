"""The 32 x 64 tile kernel by name: what the other tile kernels are tested for in
test_linear.py, test_gated.py, test_int8.py and test_cross_entropy.py, with those files'
checks and tolerances. It has the deepest ring of tiles (four stages), so parts of a
sum that begin inside a group of four passes, whose block scales come together, are
here as well, and sums shorter than the ring.
"""

from __future__ import annotations

import pytest
import torch

import sublayer_ref as R
import test_cross_entropy as CE
import test_gated as TG
import test_int8 as TI
import test_linear as TL
from gpu_util import say
from hyper_connection_residual_mhc_amd import _lib

SHORT = _lib.MHC_LINEAR_SHORT
BM, BN = 32, 64
BF16 = torch.bfloat16
# rows and columns (of a product; a gated tile has half as many) around the tiles' borders
BORDERS = ((1, 1), (BM - 1, BN - 1), (BM, BN), (BM + 1, BN + 1), (BM + 17, 3 * BN - 9), (5 * BM + 3, 2 * BN), (9 * BM, BN + 7))


def test_plans_name_it(built_library):
    from hyper_connection_residual_mhc_amd import gated as G, linear as L
    for splits in (1, 3, 64):
        want = {"kernel": SHORT, "splits": splits}
        assert L.mhc_linear_plan(40, 100, 1 << 16, 1, want) == want
        assert G.mhc_gated_plan(40, 100, 1 << 16, 1, want) == want
    # the sizes that the policy gives it, of either operator
    assert G.mhc_gated_plan(24, 14336, 7168, 4)["kernel"] == SHORT
    assert L.mhc_linear_plan(32, 7168, 4096, 6)["kernel"] == SHORT


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16", "row", "mx"])
def test_product_depths(device, kind):
    for k, K in enumerate(TL.DEPTHS):
        say(f"short product {kind} K={K}")
        TL.run_forward(device, kind, 70, 72, K, seed=k, launch={"kernel": SHORT})


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "mx"])
def test_product_tiles(device, kind):
    for k, (M, N) in enumerate(BORDERS):
        say(f"short product {kind} M={M} N={N}")
        TL.run_forward(device, kind, M, N, 192, seed=k, launch={"kernel": SHORT, "splits": 1})


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "row", "mx"])
@pytest.mark.parametrize("splits", [2, 3, 7, 64])
def test_product_splits(device, splits, kind):
    for K in (128, 1000, 2304):
        say(f"short product {kind} splits={splits} K={K}")
        TL.run_forward(device, kind, 45, 130, K, seed=splits, activation="silu", launch={"kernel": SHORT, "splits": splits})


def parts(passes):
    """Splits whose parts begin at every place of a group of four passes."""
    return (1,) if passes < 4 else (1, 2, 3, 4, passes)


@pytest.mark.gpu
def test_product_block_scales(device):
    """Scales that differ from block to block by up to 2^16, over one to thirteen passes and in parts."""
    from hyper_connection_residual_mhc_amd import linear as L
    M, N = 100, 145
    for passes in range(1, 14):
        for splits in parts(passes):
            K = 128 * passes
            say(f"short product block scales K={K} splits={splits}")
            gen = torch.Generator().manual_seed(passes)
            x, w = (torch.randn(r, K, generator=gen).to(torch.float8_e4m3fn) for r in (M, N))
            xs, ws = (torch.randint(119, 136, (r, K // 32), generator=gen, dtype=torch.uint8).view(torch.float8_e8m0fnu)
                      for r in (M, N))
            out, z = torch.empty(M, N, dtype=BF16, device=device), torch.empty(M, N, dtype=BF16, device=device)
            L.mhc_linear_fwd(x.to(device), w.to(device), out, x_scales=xs.to(device), weight_scales=ws.to(device), z=z,
                             launch={"kernel": SHORT, "splits": splits})
            torch.cuda.synchronize()
            TL.check_forward(out, z, dict(bias=None, residual=None), R.dequantise(x, xs), R.dequantise(w, ws), BF16, "none", "mx")


@pytest.mark.gpu
def test_product_rows_do_not_depend_on_the_batch(device):
    from hyper_connection_residual_mhc_amd import linear as L
    ops, *_ = TL.make("bf16", 300, 136, 1000, 6, residual=False)
    up = {k: None if v is None else v.to(device) for k, v in ops.items()}

    def run(rows):
        out = torch.empty(len(rows), 136, dtype=BF16, device=device)
        L.mhc_linear_fwd(up["x"][rows].contiguous(), up["weight"], out, bias=up["bias"], launch={"kernel": SHORT, "splits": 1})
        return out

    everything = run(list(range(300)))
    for rows in ([0], [299], [5, 150, 77], list(range(100, 229))):
        assert R.same_bytes(run(rows), everything[rows])


@pytest.mark.gpu
def test_operands_past_alignment_and_edges(device):
    """Through registers the same bytes as straight into LDS, and nothing outside the outputs and the workspace."""
    from hyper_connection_residual_mhc_amd import gated as G, linear as L
    for kind, splits in (("bf16", 1), ("mx", 3)):
        M, N, K = 45, 72, 1024
        launch = {"kernel": SHORT, "splits": splits}
        a = TL.run_forward(device, kind, M, N, K, 5, launch=launch)
        assert R.same_bytes(a, TL.run_forward(device, kind, M, N, K, 5, launch=launch, place=R.shifted))
        a = TG.run_forward(device, kind, M, N, K, 5, launch=launch)
        assert R.same_bytes(a, TG.run_forward(device, kind, M, N, K, 5, launch=launch, place=R.shifted))
        for make, sizes in ((TL.make, L.mhc_linear_fwd_workspace_bytes), (TG.make, G.mhc_gated_fwd_workspace_bytes)):
            ops = make(kind, M, N, K, 5)[0]
            at = {k: None if v is None else v.to(device) for k, v in ops.items()}
            out = R.Guarded((M, N), BF16, device)
            ws = R.Guarded((max(1, sizes(M, N, K, TG.ABI[kind], launch)),), torch.uint8, device, 0xFF)
            if make is TL.make:
                L.mhc_linear_fwd(at.pop("x"), at.pop("weight"), out.t, workspace=ws.t, launch=launch, **at)
            else:
                G.mhc_gated_fwd(at.pop("x"), at.pop("gate_weight"), at.pop("up_weight"), out.t, workspace=ws.t, launch=launch, **at)
            assert out.untouched() and ws.untouched()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16", "row", "mx", "int8"])
def test_gated_depths(device, kind):
    for k, K in enumerate(TG.DEPTHS):
        say(f"short gated {kind} K={K}")
        TG.run_forward(device, kind, 70, 36, K, seed=k, launch={"kernel": SHORT})


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "mx", "int8"])
def test_gated_tiles_and_splits(device, kind):
    for k, (M, N) in enumerate(BORDERS):
        say(f"short gated {kind} M={M} N={-(-N // 2)}")
        TG.run_forward(device, kind, M, -(-N // 2), 256, seed=k, launch={"kernel": SHORT, "splits": 1})
    for splits in (2, 3, 64):
        for K in (128, 1000, 2304):
            say(f"short gated {kind} splits={splits} K={K}")
            TG.run_forward(device, kind, 45, 70, K, seed=splits, launch={"kernel": SHORT, "splits": splits})


@pytest.mark.gpu
def test_gated_block_scales(device):
    from hyper_connection_residual_mhc_amd import gated as G
    M, N = 100, 73
    for passes in range(1, 14):
        for splits in parts(passes):
            K = 128 * passes
            say(f"short gated block scales K={K} splits={splits}")
            gen = torch.Generator().manual_seed(passes)
            codes = [torch.randn(r, K, generator=gen).to(torch.float8_e4m3fn) for r in (M, N, N)]
            scales = [torch.randint(119, 136, (r, K // 32), generator=gen, dtype=torch.uint8).view(torch.float8_e8m0fnu)
                      for r in (M, N, N)]
            out, gate, up = (torch.empty(M, N, dtype=BF16, device=device) for _ in range(3))
            c, s = [v.to(device) for v in codes], [v.to(device) for v in scales]
            G.mhc_gated_fwd(*c, out, x_scales=s[0], gate_scales=s[1], up_scales=s[2], gate=gate, up=up, activation="none",
                            launch={"kernel": SHORT, "splits": splits})
            torch.cuda.synchronize()
            TG.check_forward(out, gate, up, dict(gate_bias=None, up_bias=None),
                             [R.dequantise(v, q) for v, q in zip(codes, scales)], BF16, "none", "mx")


@pytest.mark.gpu
def test_integer_products(device):
    for k, K in enumerate((1, 7, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 520, 1279, 2048)):
        say(f"short int8 K={K}")
        TI.check(device, 70, 72, K, seed=k, launch={"kernel": SHORT})
    for k, (M, N) in enumerate(BORDERS):
        say(f"short int8 M={M} N={N}")
        TI.check(device, M, N, 384, seed=k, launch={"kernel": SHORT, "splits": 1})
    for K, splits in ((131071, 1), (131071, 5), (131056, 64)):
        say(f"short int8 K={K} splits={splits}")
        TI.check(device, 20, 40, K, 3, extreme=True, bias=False, residual=False, launch={"kernel": SHORT, "splits": splits})


@pytest.mark.gpu
def test_integer_rows_depend_on_nothing_else(device):
    a = TI.check(device, 300, 200, 1000, 7)
    for splits in (1, 2, 5):
        assert R.same_bytes(a, TI.check(device, 300, 200, 1000, 7, launch={"kernel": SHORT, "splits": splits}))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_cross_entropy(device, kind, monkeypatch):
    """Rows and columns around the tiles' and the groups' borders, and the depths."""
    monkeypatch.setitem(CE.GROUP, SHORT, 32)
    for k, (M, V) in enumerate((*BORDERS, (BM - 1, 31), (BM // 2, 32), (7, 33), (3 * BM + 5, BN // 2 + 3), (2 * BM, 2 * BN + 33))):
        say(f"short cross entropy {kind} M={M} V={V}")
        CE.run(device, kind, M, V, 192, seed=k, kernel=SHORT, reduction=("none", "mean", "sum")[k % 3])
    for k, K in enumerate((1, 7, 8, 31, 33, 63, 64, 65, 128, 129, 520, 1279)):
        say(f"short cross entropy {kind} K={K}")
        CE.run(device, kind, 45, 140, K, seed=k, kernel=SHORT, weighted=k % 2 == 0)
