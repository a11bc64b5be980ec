"""NaN and infinities in the inputs of both backward calls on the GPU reach what the
formulas let them reach, and every other output keeps its bits: each place is tried at
the first and the last row and column, and beside the places where a row's last
vector begins."""
import pytest
import torch

from error_compensated_bit_echo_amd import binding as B
from layer_reference import TYPES
from test_gpu_linear import space
from test_gpu_norm import DEV
from test_gpu_norm_forms import case, gradients, wanted

pytestmark = pytest.mark.gpu
BAD = [float("nan"), float("inf"), float("-inf")]


def planted(t, row, col, bad):
    t = t.clone()
    t[row, col] = bad
    return t


def compare(got, clean, name, rows=None, cols=None):
    """`rows` and `cols` (a list each, None for all) are the places that may differ,
    and not all of those are finite; everything else has the same bits"""
    may = torch.zeros(got.shape, dtype=torch.bool, device=DEV)
    if rows is not None or cols is not None:
        r = slice(None) if rows is None else rows
        c = slice(None) if cols is None else cols
        if rows is not None and cols is not None:
            may[torch.tensor(rows)[:, None], torch.tensor(cols)[None, :]] = True
        else:
            may[r if rows is not None else slice(None), c if cols is not None else slice(None)] = True
        assert not bool(torch.isfinite(got[may].float()).all()), f"{name}: nothing arrived"
    assert torch.equal(got[~may], clean[~may]), f"{name}: outside its rows and columns"


@pytest.mark.parametrize("H", [5, 509, 512, 1021, 2051, 4096, 8189])
@pytest.mark.parametrize("post,pre,groups", [("none", "rms", 0), ("none", "layer", 0), ("rms", "layer", 30), ("layer", "rms", 2),
                                             ("layer", "layer", 600), ("none", "rms", 1)])
def test_norm_backward(post, pre, groups, H):
    T = 600
    biases = "layer" in (post, pre)
    sums = wanted(post, pre, biases, groups > 0)
    c = case(T, H, torch.bfloat16, torch.float32, post, pre, groups, seed=7)
    clean = {n: v.clone() for n, (_, v) in gradients(c, post, pre, sums).items()}
    places = [(0, 0), (T - 1, H - 1), (77, max(H - 8, 0)), (301, max(H - 9, 0)), (300, H // 2)]
    for k, (row, col) in enumerate(places):
        bad = BAD[k % 3]
        group = [row // (T // groups)] if groups else None
        for where in ("dz", "dh_out", "y"):
            print(f"norm H={H} {post}/{pre} groups={groups} {where}[{row}, {col}] = {bad}", flush=True)
            got = gradients({**c, where: planted(c[where], row, col, bad)}, post, pre, sums)
            one, whole = [col], None  # of the row: one element, or all through the row's sums
            if where == "dz":
                dh, du = whole, whole
            elif where == "dh_out":
                dh, du = one, one
            else:
                dh, du = [], one
            dy = whole if post != "none" else du if where != "y" else []
            for n, (_, v) in got.items():
                if n == "dh":
                    reach = None if dh == [] else ([row], dh)
                elif n == "dy":
                    reach = None if dy == [] else ([row], dy)
                elif n in ("dw_pre", "db_pre"):
                    reach = ([0], one) if where == "dz" else None
                elif n == "db_post":
                    reach = ([0], du) if where != "y" else None
                elif n == "dw_post":
                    reach = ([0], du)
                else:
                    reach = (group, du)
                compare(v, clean[n], f"{where}: {n}", *(reach or ()))


# staged tiles of both sizes, direct loads, copied rows, splits, the large tiles
SIZES = [(3, 5, 7, "bf16"), (70, 90, 80, "f16"), (17, 33, 63, "bf16"), (513, 104, 4104, "bf16"), (1300, 50, 41, "f16"),
         (300, 1003, 520, "bf16"), (4090, 203, 4088, "bf16"), (203, 4090, 4086, "f16")]


@pytest.mark.parametrize("act,gated", [("none", False), ("gelu", False), ("silu", True)])
@pytest.mark.parametrize("m,n,k,dt", SIZES)
def test_linear_backward(m, n, k, dt, act, gated):
    gen = torch.Generator(device=DEV).manual_seed(m + n + k)
    rand = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(TYPES[dt])  # noqa: E731
    rows = 2 * n if gated else n
    plain = act == "none" and not gated
    c = {"dout": rand(m, n), "x": rand(m, k), "w": rand(rows, k), "p": None if plain else rand(m, rows)}
    ws = space(B.echo_linear_backward_workspace(m, n, k, act=act, gated=gated))

    def run(c):
        out = {"dx": torch.empty_like(c["x"]), "dw": torch.empty_like(c["w"]), "dbias": rand(1, rows)}
        ws.fill_(0xFF)
        B.echo_linear_backward(c["dout"], c["x"], c["w"], c["p"], out["dx"], out["dw"], dbias=out["dbias"][0], act=act,
                               gated=gated, workspace=ws)
        torch.cuda.synchronize()
        return out

    clean = run(c)
    for k2, (i, j, l) in enumerate([(0, 0, 0), (m - 1, n - 1, k - 1), (m // 2, n // 3, k // 2)]):
        bad = BAD[k2]
        both = [j, n + j] if gated else [j]
        reach = {"dout": {"dx": ([i], None), "dw": (both, None), "dbias": ([0], both)},
                 "x": {"dw": (None, [l])}, "w": {"dx": (None, [l])},
                 "p": {"dx": ([i], None), "dw": (both, None), "dbias": ([0], both)}}
        for where in ("dout", "x", "w", "p"):
            if c[where] is None:
                continue
            print(f"linear m={m} n={n} k={k} {dt} {act} gated={gated} {where} {bad}", flush=True)
            row, col = {"dout": (i, j), "x": (i, l), "w": (j, l), "p": (i, j)}[where]
            got = run({**c, where: planted(c[where], row, col, bad)})
            for name, v in got.items():
                compare(v, clean[name], f"{where}: {name}", *reach[where].get(name, ()))
