"""More cases of the paged-attention operators: batches with rows that see nothing, and queries
at the ends of their range."""
import numpy as np
import pytest

import block_scaled_fp4_sigmoid_gb300 as fm
from gpu_util import ensure_built, torch_cuda
from paged_util import Problem, check, check_codes
from oracle.formats import E4M3_TABLE

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    torch_cuda()
    ensure_built()
    from block_scaled_fp4_sigmoid_gb300 import paged_attention
    return paged_attention


def run(pa, p, t, decode=False, **more):
    if decode:
        return pa.decode_attention(t["q"], t["k_cache"], t["v_cache"], t["lens"], t["table"], **p.options(t), **more)
    return pa.prompt_attention(t["q"], t["k_cache"], t["v_cache"], t["starts"], t["lens"], t["table"], **p.options(t), **more)


def holds(pa, p, decode=False):
    want, bound = p.expected()
    t = p.tensors()
    check(run(pa, p, t, decode).double().cpu().numpy(), want, bound)
    codes, scales = run(pa, p, t, decode, fp8=True)
    check_codes(codes.cpu().numpy(), scales.cpu().numpy(), want, bound)


# ------------------------------------------------------------- pieces of work that see nothing
ROWS, LENS = [600, 500, 1], [700, 500, 33]  # 10 + 8 + 1 pieces of 64 rows, for each of 8 heads: one for each of 152 CTAs
WHOLE = {}


def whole(pa, D, fp8):
    """The sequences on their own, and what they give, checked."""
    if (D, fp8) not in WHOLE:
        p = Problem(LENS, rows=ROWS, hq=32, hkv=8, D=D, page=32, fp8=fp8, seed=60)
        t = p.tensors()
        out = run(pa, p, t)
        check(out.double().cpu().numpy(), *p.expected())
        WHOLE[D, fp8] = p, t, out, run(pa, p, t, fp8=True)
    return WHOLE[D, fp8]


def among_rows_that_see_nothing(pa, order, D, fp8):
    """order: R, the sequences above, and E, as many pieces of work that see nothing (of one row: padding, rows
    before position 0, rows past the table), as each CTA meets them, which is from the last row on."""
    import torch
    p, t, want, (codes, scales) = whole(pa, D, fp8)
    reach = p.table.shape[1] * p.page
    rows, lens, table, q, real = [], [], [], [], []
    noise = torch.randn(19, 32, D, device="cuda").bfloat16()
    for o in reversed(order):
        if o == "R":
            rows += ROWS
            lens += LENS
            table.append(t["table"])
            q.append(t["q"])
        else:
            rows += [1] * 19
            lens += [(0, -5, reach + 1 + i)[i % 3] for i in range(19)]
            table.append(t["table"][[i % 3 for i in range(19)]])
            q.append(noise)
        real += [o == "R"] * len(q[-1])
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    u = {**t, "q": torch.cat(q), "table": torch.cat(table), "lens": ints(lens), "starts": ints(np.cumsum([0] + rows).tolist())}
    real = torch.tensor(real, device="cuda")
    n = order.count("R")
    for _ in range(10):
        got = run(pa, p, u)
        assert torch.equal(got[real], want.repeat(n, 1, 1)) and not got[~real].any()
        c, s = run(pa, p, u, fp8=True)
        assert torch.equal(c[real], codes.repeat(n, 1)) and torch.equal(s[real], scales.repeat(n, 1))
        assert not c[~real].any() and not s[~real].any()
    assert fm.attn_prompt_status(torch.cuda.current_stream().cuda_stream) == (0, 0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("order", ["EER", "EERR", "EEREER", "REE"])
def test_prompt_rows_that_see_nothing_leave_the_next_queries(pa, order, D, fp8):
    """Zeros of such rows do not go where the next rows' queries are, nor the other way."""
    among_rows_that_see_nothing(pa, order, D, fp8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("order", ["ER", "ERR", "RER", "EEER", "EREER", "RERER", "RE"])
def test_prompt_rows_that_see_nothing_leave_the_roles_in_step(pa, order, D, fp8):
    """An odd number of such pieces before others, between and behind them."""
    among_rows_that_see_nothing(pa, order, D, fp8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_with_one_padding_row(pa, D, fp8):
    """2560 rows and one of padding: some CTAs meet a piece that sees nothing first, others do not."""
    import torch
    p = Problem([2560, 0], rows=[2560, 1], hq=32, hkv=8, D=D, page=64, fp8=fp8, seed=61)
    t = p.tensors()
    alone = {**t, "q": t["q"][:-1], "lens": t["lens"][:1], "starts": t["starts"][:2], "table": t["table"][:1]}
    want = run(pa, p, alone)
    for _ in range(5):
        got = run(pa, p, t)
        assert torch.equal(got[:-1], want) and not got[-1].any()
    # among the first rows are those that a CTA takes after the padding: in 64 bits
    p.starts, p.lens, p.table, p.q = np.array([0, 256]), np.array([256]), p.table[:1], p.q[:256]
    check(got[:256].double().cpu().numpy(), *p.expected())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_with_rows_before_the_first_position(pa, D, fp8):
    """Pieces wholly before position 0, partly, and ordinary ones, as 60 sequences bring them."""
    import torch
    rng = np.random.default_rng(62)
    rows = rng.integers(1, 150, 60)
    lens = np.where(rng.random(60) < 0.5, rng.integers(0, 60, 60), rows + rng.integers(0, 100, 60))
    p = Problem(lens.tolist(), rows=rows.tolist(), hq=16, hkv=4, D=D, page=16, fp8=fp8, seed=62)
    t = p.tensors()
    want, bound = p.expected()
    got = run(pa, p, t)
    check(got.double().cpu().numpy(), want, bound)
    for _ in range(10):
        assert torch.equal(run(pa, p, t), got)
    assert fm.attn_prompt_status(torch.cuda.current_stream().cuda_stream) == (0, 0)


@pytest.mark.parametrize("hq,hkv,D", [(32, 8, 64), (32, 8, 128), (48, 16, 128)])
def test_prompt_outputs_staged_before_the_next_queries(pa, hq, hkv, D):
    """E4M3 caches, five and more short pieces a CTA: each one's outputs leave by the memory that the next one's queries
    arrive in.  bf16 and codes, the same every time."""
    import torch
    rows = [62 - i % 3 for i in range(100)]
    p = Problem([n + 5 * i % 40 for i, n in enumerate(rows)], rows=rows, hq=hq, hkv=hkv, D=D, page=16, fp8=True, seed=63)
    t = p.tensors()
    want, bound = p.expected()
    got, (codes, scales) = run(pa, p, t), run(pa, p, t, fp8=True)
    check(got.double().cpu().numpy(), want, bound)
    check_codes(codes.cpu().numpy(), scales.cpu().numpy(), want, bound)
    for _ in range(100):
        assert torch.equal(run(pa, p, t), got)
        c, s = run(pa, p, t, fp8=True)
        assert torch.equal(c, codes) and torch.equal(s, scales)
    assert fm.attn_prompt_status(torch.cuda.current_stream().cuda_stream) == (0, 0)


# ------------------------------------------------------------- queries at the ends of their range, and beyond
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_prompt_queries_that_are_not_finite_and_see_nothing(pa, D, value):
    """E4M3 caches: rows before position 0 and rows over holes only, in a tile with others that see something, are
    zeros whatever their queries hold."""
    p = Problem([40, 60], rows=[60, 60], hq=8, hkv=2, D=D, page=16, fp8=True, seed=50)
    p.table[1, 0] = -1  # positions 0 .. 15 of the second sequence
    blind = np.r_[0:20, 60:76]
    p.q[blind, :, 3] = value
    t = p.tensors()
    p.q[blind] = 0
    want, bound = p.expected()
    assert (want[blind] == 0).all()
    check(run(pa, p, t).double().cpu().numpy(), want, bound)
    codes, scales = run(pa, p, t, fp8=True)
    check_codes(codes.cpu().numpy(), scales.cpu().numpy(), want, bound)
    assert not (codes.cpu().numpy()[blind] & 0x7F).any()


@pytest.mark.parametrize("D,n", [(64, 60), (128, 60), (128, 5000)])
def test_prompt_infinite_queries(pa, D, n):
    """E4M3 caches (5000: in parts): q holds one infinity, against keys whose value there is of one
    sign.  Scores are all -infinity: zeros; all +infinity: NaN.  The other rows are what they are."""
    p = Problem([n, n], rows=[30, 30], hq=8, hkv=2, D=D, page=16, fp8=True, seed=51)
    p.kc[..., 3] = np.where((p.kc[..., 3] & 0x7F) == 0x7F, p.kc[..., 3], 0x28)
    p.k = E4M3_TABLE[p.kc] * p.ks.astype(np.float64)[:, None, None]
    p.q[[4, 40], :, 3], p.q[[5, 41], :, 3] = -np.inf, np.inf
    t = p.tensors()
    got = run(pa, p, t).double().cpu().numpy()
    finite = np.delete(np.arange(60), [4, 5, 40, 41])
    p.q[[4, 5, 40, 41]] = 0
    want, bound = p.expected()
    check(got[finite], want[finite], bound[finite])
    assert (got[[4, 40]] == 0).all() and np.isnan(got[[5, 41]]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("power", [118, 104, -104, -118])
def test_queries_near_the_ends_of_the_range(pa, power, decode, D, fp8):
    """Queries of 2^power against keys of 2^-power: ordinary scores."""
    rows = [1, 1, 1] if decode else [60, 17, 1]
    p = Problem([600, 17, 130], rows=rows, hq=8, hkv=2, D=D, page=16, fp8=fp8, k_size=2.0 ** -power, seed=52)
    p.q *= 2.0 ** power
    holds(pa, p, decode)


@pytest.mark.parametrize("D,n", [(64, 60), (128, 60), (128, 40000)])
def test_decode_infinite_queries(pa, D, n):
    """As above for decode, beside a large value, which is nothing next to an infinity."""
    p = Problem([n, n], hq=8, hkv=2, D=D, page=16, fp8=True, seed=54)
    p.kc[..., 3] = np.where((p.kc[..., 3] & 0x7F) == 0x7F, p.kc[..., 3], 0x28)
    p.q[0, :, 3], p.q[1, :, 3] = -np.inf, np.inf
    p.q[:, :, 4] = -3e38
    got = run(pa, p, p.tensors(), True).double().cpu().numpy()
    assert (got[0] == 0).all() and np.isnan(got[1]).all()
