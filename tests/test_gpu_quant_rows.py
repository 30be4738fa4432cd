"""qknorm_quant_rows on the GPU against its definition in 64 bits: the same integers and the same scale."""
import math

import pytest
import torch

import qk_norm_amd as q
from lowbit_ref import quant_rows

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


def _run(x, ldq=None):
    T, n = x.shape
    space = torch.full((T, ldq or n), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((T,), -1.0, device="cuda")
    q.qknorm_quant_rows(x, space[:, :n], scale)
    torch.cuda.synchronize()
    assert bool((space[:, n:] == 99).all()), "values past the rows' ends were written"
    return space[:, :n].cpu(), scale.cpu()


def _check(x, got):
    want, ws = quant_rows(x)
    assert torch.equal(got[0], want)
    assert torch.equal(torch.nan_to_num(got[1], nan=-7.0), torch.nan_to_num(ws, nan=-7.0))


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "f16"])
@pytest.mark.parametrize("T,n", [(1, 16), (3, 48), (5, 512), (4, 528), (7, 2048), (2, 2064), (3, 4096), (2, 4112),
                                 (1, 8192), (2, 12304), (1, 16384), (2, 16400), (1, 40000)])
def test_against_definition(T, n, dtype):
    print(f"[quant] T={T} n={n} {dtype}", flush=True)
    g = torch.Generator().manual_seed(T * 100003 + n)
    x = (torch.randn(T, n, generator=g) * torch.exp2(torch.randn(T, 1, generator=g) * 4)).to(dtype).cuda()
    _check(x, _run(x))


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "f16"])
def test_halfway_points_and_their_neighbours(dtype):
    # rows whose maximum is 127 * 2^e: x = (m + .5) * 2^e is halfway between integers
    rows = []
    for e in (-8, 0, 6):
        half = torch.arange(-126.5, 127.0, 1.0)
        r = torch.cat([torch.tensor([127.0]), half, half * (1 + 2.0 ** -7), half * (1 - 2.0 ** -7)])
        r = r.clamp(-127, 127)[:640]
        rows.append(torch.cat([r, torch.zeros(640 - len(r))]) * 2.0 ** e)
    # half of any maximum is 63.5 steps
    g = torch.Generator().manual_seed(5)
    for _ in range(64):
        top = (torch.rand(1, generator=g) + 1).to(dtype).float()
        rows.append(torch.cat([top, top / 2, -top / 2, torch.rand(637, generator=g) * top]))
    x = torch.stack(rows).to(dtype).cuda()
    print("[quant] halfway", flush=True)
    _check(x, _run(x))


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "f16"])
def test_rows_of_zeros_extremes_and_non_finite_values(dtype):
    big = float(torch.finfo(dtype).max)
    x = torch.zeros(8, 64)
    x[1, 3] = big
    x[1, 4] = -big / 2
    x[2, :] = 2.0 ** -24
    x[3, 5], x[3, 6] = math.inf, 1.0
    x[4, 7], x[4, 8] = math.nan, 2.0
    x[5, 9] = -math.inf
    x[6] = 2.0 ** -120 if dtype == torch.bfloat16 else 2.0 ** -14
    x[7] = 2.0 ** -99 if dtype == torch.bfloat16 else 2.0 ** -23
    print("[quant] extremes", flush=True)
    xt = x.to(dtype).cuda()
    got = _run(xt)
    _check(xt, got)
    assert got[1][3].isnan() and got[1][4].isnan() and got[1][5].isnan() and got[1][0] == 0


def test_pitches_and_many_rows():
    g = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn(2051, 1024 + 40, generator=g, device="cuda").to(torch.bfloat16)
    x = wide[:, 8:1032]
    print("[quant] pitches", flush=True)
    _check(x, _run(x, ldq=1040))


def test_past_four_gib():
    # the last rows of an input whose rows lie 32 MiB apart, and of an output 48 MiB apart
    T, n = 140, 64
    wide = torch.empty(T, 1 << 24, dtype=torch.float16, device="cuda")
    out = torch.empty(T, 48 << 20, dtype=torch.int8, device="cuda")
    g = torch.Generator().manual_seed(11)
    x = torch.randn(T, n, generator=g).to(torch.float16)
    wide[:, :n] = x.cuda()
    scale = torch.empty(T, device="cuda")
    print("[quant] past 4 GiB", flush=True)
    q.qknorm_quant_rows(wide[:, :n], out[:, :n], scale)
    torch.cuda.synchronize()
    want, ws = quant_rows(x)
    assert torch.equal(out[:, :n].cpu(), want) and torch.equal(scale.cpu(), ws)


def test_empty():
    q.qknorm_quant_rows(torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"),
                        torch.empty(0, 32, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"))
