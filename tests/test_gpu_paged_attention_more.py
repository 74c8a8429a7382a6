"""More cases of the paged-attention operators: batches with rows that see nothing, queries
at the ends of their range, and weights far below the largest."""
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


# ------------------------------------------------------------- weights far below the largest
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [0, 1, 1000])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("first", [True, False])
def test_many_small_weights_below_a_large_one(pa, D, rows, first, fp8):
    """One token stands out by 2^25.5 and its value is 0, those of the other 131071 are 1: together they make 0.3 % of a row.
    rows 0: decode; 1: a prompt in parts; 1000: whole.  A weight is off by 2^-11 of it in fp16 and 2^-8 in bf16, and in fp16
    by half a step of its smallest, 2^-25, where weights are scaled by 2^7 or more: 2^-32 of the largest for each token.  The sums' chains, of
    2^13 steps at most, are off by 2^-23 a step; the exponent by three roundings of up to 25.5; the result by 2^-8."""
    import torch
    page, n = 128, 1 << 17
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    k, v = torch.zeros(2, 2, 1, page, D, device="cuda")
    at = 5 if first else page - 7
    k[1, 0, at, 0] = 1.0
    v += 1.0
    v[1, 0, at] = 0.0
    k, v = k.to(dt), v.to(dt)
    scale = {x: torch.ones(1, device="cuda") for x in ("k_scale", "v_scale")} if fp8 else {}
    hq, T = 4, max(rows, 1)
    cols = n // page + 2
    table = torch.zeros((1, cols), dtype=torch.int32, device="cuda")
    table[0, 0 if first else n // page - 1] = 1
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    q = torch.zeros(T, hq, D, device="cuda").bfloat16()
    q[:, :, 0] = 1.0
    s = 25.5 * np.log(2.0)
    if rows:
        got = pa.prompt_attention(q, k, v, starts, lens, table, scale=s, **scale)
    else:
        got = pa.decode_attention(q, k, v, lens, table, scale=s, **scale)
    got = got.double().cpu().numpy()
    # (a row that the token which stands out comes after sees even ones only)
    p = n - T + np.arange(T)
    seen = p >= (at if first else n - page + at)
    others = p + 1 - seen
    small = 2.0 ** -25.5 * others
    want = np.where(seen, small / (1 + small), 1.0)[:, None, None]
    lost = others * 2.0 ** -32 * fp8
    tol = want * (2.0 ** -8 + (2.0 ** -11 if fp8 else 2.0 ** -8) + 2.0 ** -10 + 3 * 25.5 * 2.0 ** -24) + (lost * seen)[:, None, None]
    assert (np.abs(got - want) <= tol).all(), (got[:, 0, 0], want[:, 0, 0])


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("v_size", [1e-33, 1e30])
def test_scales_of_values_far_from_one(pa, decode, v_size):
    """E4M3 caches, the scale of V near the ends of fp32: the sums' own scale does not meet it in one number."""
    p = Problem([3000, 90], rows=[1, 1] if decode else [70, 90], hq=8, hkv=2, D=64, page=16, fp8=True, seed=53)
    p.vs = (p.vs * v_size).astype(np.float32)
    p.v = E4M3_TABLE[p.vc] * p.vs.astype(np.float64)[:, None, None]
    want, bound = p.expected()
    check(run(pa, p, p.tensors(), decode).double().cpu().numpy(), want, bound)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,n,rows", [(1, 700, 1), (300, 90, 1), (3, 9000, 1), (3, 9000, 20), (1, 700, 500)])
def test_small_weights_beside_large_ones_everywhere(pa, B, n, rows, D, fp8):
    """In each 16 tokens one stands out by 2^25.5 and has no value, the others have all: what they give is small, and
    known as well as above (decode: half a step of 2^-24 of weights scaled by 2^15, 2^-40)."""
    import torch
    page = 32
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    k, v = torch.zeros(2, 1, 1, page, D, device="cuda")
    k[:, :, ::16, 0] = 1.0
    v += 1.0
    v[:, :, ::16] = 0.0
    k, v = k.to(dt), v.to(dt)
    scale = {x: torch.ones(1, device="cuda") for x in ("k_scale", "v_scale")} if fp8 else {}
    table = torch.zeros((B, -(-n // page)), dtype=torch.int32, device="cuda")
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda") * rows
    q = torch.zeros(B * rows, 4, D, device="cuda").bfloat16()
    q[:, :, 0] = 1.0
    s = 25.5 * np.log(2.0)
    if rows > 1:
        got = pa.prompt_attention(q, k, v, starts, lens, table, scale=s, **scale)
    else:
        got = pa.decode_attention(q, k, v, lens, table, scale=s, **scale)
    seen = n - rows + 1 + np.arange(rows)
    large = (seen + 15) // 16
    want = (seen - large) * 2.0 ** -25.5 / (large + (seen - large) * 2.0 ** -25.5)
    lost = (seen - large) / large * (2.0 ** -32 if rows > 1 else 2.0 ** -40) * fp8
    tol = want * (2.0 ** -8 + (2.0 ** -11 if fp8 else 2.0 ** -8) + 2.0 ** -10 + 3 * 25.5 * 2.0 ** -24) + lost
    got = got.double().cpu().numpy().reshape(B, rows, -1)
    assert (np.abs(got - want[:, None]) <= tol[:, None]).all(), (got[0, :, 0], want)


# ------------------------------------------------------------- calls that the header allows
@pytest.mark.parametrize("fp8", [False, True])
def test_prompts_in_a_captured_graph_follow_their_tensors(pa, fp8):
    """Prompts of a padded batch, captured once and replayed as sequences and rows change (a sequence that was padding
    gets tokens, another one ends), over one workspace in two graphs."""
    import torch
    rng = np.random.default_rng(70)
    ps = []
    for lens, rows in (([900, 0, 700, 0], [30, 1, 60, 9]), ([0, 300, 2500, 5], [1, 90, 8, 1]), ([0, 0, 0, 0], [25, 25, 25, 25])):
        p = Problem(lens, rows=rows, hq=16, hkv=4, D=64, page=32, fp8=fp8, seed=71)
        p.q = p.q[:100]
        ps.append(p)
    k, v = (torch.zeros((200, 4, 32, 64), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda") for _ in range(2))
    q, out = (torch.zeros((100, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lens, starts, table = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((4,), (5,), (4, 90)))
    ks, vs = (torch.ones(4, device="cuda") for _ in range(2)) if fp8 else (None, None)
    ws = torch.empty(pa.prompt_workspace_size(k, 16), dtype=torch.uint8, device="cuda")

    def call():
        pa.prompt_attention(q, k, v, starts, lens, table, k_scale=ks, v_scale=vs, ws=ws, out=out)

    call()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for i in range(6):
        p = ps[i % 3]
        t = p.tensors()
        n = len(p.q)
        q[:n] = t["q"]
        k[:p.pages], v[:p.pages] = t["k_cache"], t["v_cache"]
        table.fill_(-1)
        table[:, :p.table.shape[1]] = t["table"]
        lens.copy_(t["lens"])
        starts.copy_(t["starts"])
        if fp8:
            ks.copy_(t["k_scale"])
            vs.copy_(t["v_scale"])
        out.fill_(7)
        graphs[i % 2].replay()
        want, bound = p.expected()
        got = out.double().cpu().numpy()
        check(got[:n], want, bound)
        assert (got[n:] == 7).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (1, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1), (0, 2 ** 31 - 1)])
def test_the_largest_windows_and_sinks(pa, window, sinks, decode, fp8):
    rows = [1, 1, 1] if decode else [70, 3, 130]
    holds(pa, Problem([300, 3, 2000], rows=rows, hq=8, hkv=2, D=128, page=32, fp8=fp8, window=window, sinks=sinks, seed=72), decode)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("value", [2 ** 31 - 1, -2 ** 31])
def test_lengths_that_are_no_lengths(pa, value, fp8):
    """Lengths past the table and below zero: zeros, nothing is stored, and the other sequences are what they are."""
    import torch
    p = Problem([300, 40, 130], rows=[1, 1, 1], hq=8, hkv=2, D=64, page=16, fp8=fp8, seed=73)
    t = p.tensors()
    q = t["q"]
    for prompt in (False, True):
        want = run(pa, p, t, not prompt)
        lens = t["lens"].clone()
        lens[1] = value
        got = run(pa, p, {**t, "lens": lens}, not prompt)
        assert not got[1].any() and torch.equal(got[[0, 2]], want[[0, 2]])
    new = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    rope = torch.ones(p.table.shape[1] * p.page, 64, device="cuda")
    k, v = t["k_cache"].clone(), t["v_cache"].clone()
    one, three = torch.full_like(q, 7), torch.full_like(q, 7)
    more = {"k_scale": t["k_scale"], "v_scale": t["v_scale"]}
    pa.append_kv(q, new, new, rope, k, v, lens, t["table"], q_out=one, **more)
    assert not one[1].any()
    lens[1] = 0
    pa.append_kv(q, new, new, rope, t["k_cache"], t["v_cache"], lens, t["table"], q_out=three, **more)
    assert torch.equal(one, three)
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # noqa: E731
    assert same(k, t["k_cache"]) and same(v, t["v_cache"])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_rows_in_front_of_the_first_sequence(pa, D, fp8):
    """starts that begin behind row 0, queries that are ranges of wider rows."""
    import torch
    p = Problem([200, 0, 90], rows=[70, 3, 90], hq=8, hkv=2, D=D, page=16, fp8=fp8, seed=74)
    t = p.tensors()
    want = run(pa, p, t)
    wide = torch.full((p.T + 9, 12, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[5:5 + p.T, 2:10] = t["q"]
    out = torch.full((p.T + 9, 8, D), 7.0, dtype=torch.bfloat16, device="cuda")
    run(pa, p, {**t, "q": wide[:, 2:10], "starts": t["starts"] + 5}, out=out)
    assert torch.equal(out[5:5 + p.T], want) and (out[:5] == 7).all() and (out[5 + p.T:] == 7).all()


@pytest.mark.parametrize("R", [0, 64])
@pytest.mark.parametrize("fp8", [False, True])
def test_sublayer_of_a_padded_batch(pa, R, fp8):
    """Padding rows, which hold NaN, leave the other rows what they are, and are what the output product makes of zeros."""
    import torch
    torch.manual_seed(75)
    H, hq, hkv, D, page, B = 512, 16, 4, 64, 16, 30
    w = lambda m, n: (torch.randint(0, 120, (m, n), device="cuda").to(torch.uint8), torch.rand(-(-m // 128), -(-n // 128), device="cuda") * 1e-3)  # noqa: E731
    gamma = torch.ones(H, device="cuda").bfloat16()
    a = torch.rand(12 * page, R // 2, device="cuda")
    scales = {"k_scale": torch.full((hkv,), 0.1, device="cuda"), "v_scale": torch.full((hkv,), 0.1, device="cuda")} if fp8 else {}
    layer = pa.Fp8BlockAttention(gamma, *w((hq + 2 * hkv) * D, H), *w(H, hq * D), hq, hkv, D,
                                 torch.cat((a.cos(), a.sin()), 1) if R else None, **scales)
    table = torch.randperm(B * 12, device="cuda").view(B, 12).int()
    rows = [100 + i for i in range(15)] + [1 + i % 3 for i in range(15)]
    lens = torch.tensor([n if i < 15 else 0 for i, n in enumerate(rows)], dtype=torch.int32, device="cuda")
    starts = torch.tensor(np.cumsum([0] + rows), dtype=torch.int32, device="cuda")
    n, T = int(starts[15]), int(starts[-1])
    x, r = (torch.randn(T, H, device="cuda").bfloat16() for _ in range(2))
    x[n:] = float("nan")
    new = lambda: torch.zeros(B * 12, hkv, page, D, device="cuda").to(torch.float8_e4m3fn if fp8 else torch.bfloat16)  # noqa: E731
    (k, v), (k2, v2) = (new(), new()), (new(), new())
    want, _ = layer.forward(x[:n], r[:n], k, v, lens[:15], table[:15], starts[:16])
    for _ in range(5):
        got, _ = layer.forward(x, r, k2, v2, lens, table, starts)
        assert torch.equal(got[:n], want) and not got[n:].any()
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # noqa: E731
    assert same(k, k2) and same(v, v2)
