"""The layers beside the gated delta rule (head norms with rotation, linear
attention, the 4-bit cache and its attention) against float64 definitions."""
import math

import pytest
import torch

from tests import layers_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def rt():
    from linear_attn_decode_pace_amd import runtime
    return runtime


def randn(shape, g, dtype=F32):
    return torch.randn(shape, generator=g).to(dtype)


def bits(x):
    return x.contiguous().view(torch.int16 if x.dtype == BF16 else torch.int32)


# ---- head norms with rotation ------------------------------------------------

def norm_bound(y, dtype, d):
    """Per element.  The sum of squares is within (d / 64 + 7) roundings, half
    of that in its root; the quotient, weight, scale and the two products of
    the rotation add 8; the reduced angle is within 2^-24 turns (4e-7 rad,
    6.3 roundings) and sine and cosine within 4: at most (d / 128 + 22) u of
    the row's largest channel pair, and the final rounding."""
    top = y.abs().amax(-1, keepdim=True) * math.sqrt(2)
    return (d / 128 + 22) * ref.U32 * top + ref.HALF_STEP[dtype] * y.abs() * 1.001


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,hq,hk,d,norm,rot,adjacent", [
    (1, 1, 0, 128, "l2", 0, False),
    (5, 16, 16, 128, "l2", 0, False),
    (33, 32, 8, 128, "rms", 64, False),
    (7, 4, 2, 128, "rms", 128, False),
    (9, 4, 3, 128, "rms", 128, True),
    (6, 3, 1, 256, "rms", 64, True),
    (13, 5, 2, 80, "rms", 20, False),
    (13, 5, 2, 80, "l2", 40, True),
    (4, 2, 2, 96, "none", 96, False),
    (3, 7, 1, 64, "rms", 32, False),
    (11, 3, 2, 33, "rms", 10, False),
    (5, 2, 1, 1, "l2", 0, False),
    (2, 1, 1, 1024, "rms", 1024, False),
    (3, 2, 1, 1000, "rms", 334, True),
])
def test_norm_rope(tokens, hq, hk, d, norm, rot, adjacent, dtype):
    g = ref.gen(tokens * 1000 + d)
    rows = randn((tokens, (hq + hk) * d + 24), g, dtype) * 3
    q, k = rows[:, :hq * d].view(tokens, hq, d), rows[:, hq * d:(hq + hk) * d].view(tokens, hk, d)
    qw, kw = (1 + 0.2 * randn((d,), g), 1 + 0.2 * randn((d,), g)) if norm == "rms" else (None, None)
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g, dtype=torch.int32)
    pos[0], pos[-1] = 0, 2 ** 31 - 1
    freq = torch.exp(-math.log(10000.0) * torch.arange(rot // 2) / max(1, rot // 2)).float() if rot else None
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    rows_d = rows.cuda()
    qd, kd = rows_d[:, :hq * d].view(tokens, hq, d), rows_d[:, hq * d:(hq + hk) * d].view(tokens, hk, d)
    qo, ko = rt().qk_norm_rope(qd, kd if hk else None, norm, dev(qw), dev(kw), 1e-5, 0.37,
                               dev(pos), dev(freq), adjacent)
    for got, x, w, s in ((qo, q, qw, 0.37), (ko, k, kw, 1.0))[:2 if hk else 1]:
        y = ref.norm_rope(x, norm, w, 1e-5, pos, freq, adjacent, s)
        assert got.dtype == dtype and got.is_contiguous()
        off = (got.cpu().double() - y).abs()
        assert (off <= norm_bound(y, dtype, d)).all(), float((off / norm_bound(y, dtype, d)).max())
    if hk == 0:
        assert ko is None
    assert torch.equal(bits(rows_d.cpu()), bits(rows))       # inputs as they were


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,hq,hk,d,norm,rot,adjacent", [
    (19, 5, 3, 96, "rms", 24, False),                  # vectors of every width
    (19, 3, 8, 80, "none", 40, True),
    (6, 2, 1, 72, "l2", 8, False),
    (6, 2, 1, 100, "rms", 36, False),
    (300, 1, 1, 80, "rms", 20, False),
    (1100, 4, 2, 104, "l2", 56, True),
])
def test_norm_rope_widths(tokens, hq, hk, d, norm, rot, adjacent, dtype):
    test_norm_rope(tokens, hq, hk, d, norm, rot, adjacent, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,rot,adjacent", [(128, 64, False), (80, 20, False), (256, 256, True), (33, 0, False)])
def test_norm_in_place_and_unaligned_rows(d, rot, adjacent, dtype):
    g = ref.gen(d)
    freq = torch.exp(-torch.arange(rot // 2) / 7.0).float().cuda() if rot else None
    pos = torch.randint(0, 5000, (19,), generator=g, dtype=torch.int32).cuda()
    x, y = randn((19, 3, d), g, dtype).cuda(), randn((19, 2, d), g, dtype).cuda()
    want = rt().qk_norm_rope(x, y, "l2", pos=pos, inv_freq=freq, adjacent=adjacent)
    odd = torch.empty(19 * (5 * d + 1) + 1, dtype=dtype, device="cuda")[1:]
    rows = odd.view(19, 5 * d + 1)
    qv, kv = rows[:, :3 * d].view(19, 3, d), rows[:, 3 * d:5 * d].view(19, 2, d)
    qv.copy_(x), kv.copy_(y)
    got = rt().qk_norm_rope(qv, kv, "l2", pos=pos, inv_freq=freq, adjacent=adjacent)
    for a, b in zip(got, want):     # another order of the sum of squares: a few roundings
        assert torch.allclose(a.float(), b.float(), rtol=2 ** -7 if dtype == BF16 else 32 * ref.U32, atol=1e-6)
    rt().qk_norm_rope(x, y, "l2", pos=pos, inv_freq=freq, adjacent=adjacent, q_out=x, k_out=y)
    assert torch.equal(bits(x), bits(want[0])) and torch.equal(bits(y), bits(want[1]))


def test_norm_zero_rows_and_zero_tokens():
    x = torch.zeros((3, 2, 64), device="cuda")
    q, _ = rt().qk_norm_rope(x, norm="rms", eps=1e-6)
    assert (q == 0).all()
    q, k = rt().qk_norm_rope(x[:0], x[:0])
    assert q.shape == (0, 2, 64) and k.shape == (0, 2, 64)


# ---- linear attention ----------------------------------------------------------

def linear_inputs(seed, t, b, h, dk, dv, dtype, ragged, start):
    g = ref.gen(seed)
    q = torch.nn.functional.normalize(randn((t, b, h, dk), g), dim=-1).to(dtype)
    k = torch.nn.functional.normalize(randn((t, b, h, dk), g), dim=-1).to(dtype)
    v = randn((t, b, h, dv), g, dtype)
    decay = torch.exp(-torch.exp2(-8.0 * torch.arange(1, h + 1) / h)).float()
    decay[0] = 1.0
    if h > 2:
        decay[1] = 0.0
    lens = None
    if ragged:
        lens = torch.randint(0, t + 1, (b,), generator=g, dtype=torch.int32)
        lens[0], lens[-1] = t + 5, 0                   # clamped to t; nothing
        if b > 2:
            lens[1] = 1
    state = 0.3 * randn((b, h, dk, dv), g) if start else None
    return q, k, v, decay, state, lens


def check_linear(got, state_got, want, state_want, sentinel):
    """Relative 2-norm of each (sequence, head).  A float32 sum of n terms is
    off by at most n u times its terms' sum, about sqrt(n) u in the 2-norm of
    independent roundings; with up to 2048 tokens and 128 + 64 terms a chunk
    100 u = 6e-6 is several times what those give."""
    live = ~torch.isnan(want)
    assert (got[~live] == sentinel).all()
    for name, a, b in (("out", torch.where(live, got, 0.0), torch.where(live, want, 0.0)),
                       ("state", state_got, state_want)):
        dims = (0, 3) if name == "out" else (2, 3)
        off = torch.linalg.vector_norm(a - b, dim=dims)
        size = torch.linalg.vector_norm(b, dim=dims)
        assert (off <= 100 * ref.U32 * size).all(), (name, float((off / size.clamp(min=1e-30)).max()))


@pytest.mark.parametrize("t,b,h,dk,dv,dtype,ragged,start", [
    (1, 1, 1, 64, 16, BF16, False, False),
    (1, 5, 3, 128, 128, BF16, False, True),
    (1, 3, 2, 64, 48, F32, True, True),
    (2, 2, 3, 128, 256, BF16, False, True),
    (16, 3, 2, 64, 64, BF16, True, True),
    (17, 3, 3, 128, 128, BF16, True, True),
    (63, 2, 2, 64, 128, BF16, False, True),
    (64, 2, 2, 128, 64, BF16, False, False),
    (65, 2, 3, 128, 128, BF16, True, True),
    (130, 4, 3, 128, 16, BF16, True, False),
    (200, 2, 2, 64, 240, BF16, True, True),
    (129, 2, 2, 128, 256, BF16, False, True),
    (700, 1, 3, 128, 128, BF16, False, True),
    (1030, 3, 1, 64, 64, BF16, True, True),
    (2048, 1, 1, 128, 128, BF16, False, False),
    (40, 2, 2, 128, 96, F32, True, True),
    (257, 1, 3, 64, 128, F32, False, False),
])
def test_linear_attention(t, b, h, dk, dv, dtype, ragged, start):
    q, k, v, decay, state, lens = linear_inputs(t + dv, t, b, h, dk, dv, dtype, ragged, start)
    want, end = ref.linear(q, k, v, decay, state, lens, dk ** -0.5)
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    out = torch.full((t, b, h, dv), 7.0, device="cuda")
    args = [x.cuda() for x in (q, k, v, decay)]
    got, state_got = rt().linear_attention(*args, state=dev(state), lens=dev(lens), scale=dk ** -0.5, out=out)
    assert got is out
    check_linear(got.cpu().double(), state_got.cpu().double(), want, end, 7.0)
    # in place, and bit for bit the same
    if start:
        s = state.cuda()
        again = torch.full_like(out, 7.0)
        _, s2 = rt().linear_attention(*args, state=s, lens=dev(lens), scale=dk ** -0.5, out=again, state_out=s)
        assert s2 is s and torch.equal(bits(s), bits(state_got)) and torch.equal(bits(again), bits(got))


@pytest.mark.parametrize("t,b,h,dk,dv,ragged,start", [
    (17, 3, 3, 128, 128, True, True),                  # shorter than one chunk of 32
    (32, 2, 2, 64, 64, False, True),
    (33, 2, 3, 128, 240, True, True),
    (64, 2, 2, 64, 16, False, False),
    (95, 3, 3, 128, 64, True, True),
    (700, 1, 3, 128, 128, False, True),                # segments
    (1030, 3, 1, 64, 208, True, True),
    (2048, 1, 1, 128, 256, False, False),
    (70, 64, 5, 128, 128, True, True),                 # wide column blocks
    (37, 43, 6, 64, 240, True, False),
])
def test_linear_attention_float32_prompts(t, b, h, dk, dv, ragged, start):
    test_linear_attention(t, b, h, dk, dv, F32, ragged, start)
    q, k, v, decay, state, lens = linear_inputs(t, t, b, h, dk, dv, F32, True, start)
    dev = [x.cuda() for x in (q, k, v, decay)]
    state = None if state is None else state.cuda()
    one = rt().linear_attention(*dev, state=state, lens=lens.cuda(), out=torch.zeros(v.shape, device="cuda"))
    for i in range(b):                                 # what stands behind the end is not read
        for x in dev[:3]:
            x[min(int(lens[i]), t):, i] = math.nan
    two = rt().linear_attention(*dev, state=state, lens=lens.cuda(), out=torch.zeros(v.shape, device="cuda"))
    for x, y in zip(one, two):
        assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,b,h,dk,dv,ragged,start", [
    (1, 7, 3, 128, 48, True, True),                    # column blocks that share lines of the state
    (1, 3, 3, 64, 112, False, False),
    (2, 5, 1, 128, 80, True, True),
    (7, 3, 5, 64, 192, True, True),
    (8, 4, 2, 128, 32, False, True),
    (9, 4, 3, 128, 16, True, True),
    (15, 1, 1, 64, 96, False, False),
    (16, 9, 3, 128, 128, True, True),
])
def test_linear_attention_steps_of_odd_widths(t, b, h, dk, dv, ragged, start, dtype):
    """Per element.  A state element is a sum over tokens whose terms pass at
    most t roundings of a product with g and t of a sum, so it is off by at most
    2 t u of the same sum over absolute values; an output adds d_k products of
    it, one rounding each, in some order, and the scale: (2 t + d_k + 8) u of the
    same formula over absolute values, rigorous to first order in u.  (Relative to the
    result itself no bound holds: one token's output is (q . k) v, and a
    product q . k of unit vectors can cancel to anything.)"""
    q, k, v, decay, state, lens = linear_inputs(t + dv, t, b, h, dk, dv, dtype, ragged, start)
    want, end = ref.linear(q, k, v, decay, state, lens, dk ** -0.5)
    size = lambda x: None if x is None else x.abs()  # noqa: E731
    mass, end_mass = ref.linear(size(q), size(k), size(v), decay, size(state), lens, dk ** -0.5)
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    out = torch.full((t, b, h, dv), 7.0, device="cuda")
    args = [x.cuda() for x in (q, k, v, decay)]
    got, state_got = rt().linear_attention(*args, state=dev(state), lens=dev(lens), scale=dk ** -0.5, out=out)
    got, state_got = got.cpu().double(), state_got.cpu().double()
    live = ~torch.isnan(want)
    assert (got[~live] == 7.0).all()
    assert ((got - want).abs()[live] <= ((2 * t + dk + 8) * ref.U32 * mass)[live]).all()
    assert ((state_got - end).abs() <= 2 * t * ref.U32 * 1.001 * end_mass).all()


@pytest.mark.parametrize("t,b,h,dk,dv,ragged,start", [
    (70, 64, 5, 128, 128, True, True),                 # states enough for wide column blocks
    (37, 43, 6, 64, 240, True, False),
    (600, 12, 5, 64, 128, True, True),                 # and of segments
    (520, 3, 21, 128, 128, False, True),
    (1300, 2, 8, 128, 64, True, False),
])
def test_linear_attention_of_many_states(t, b, h, dk, dv, ragged, start):
    test_linear_attention(t, b, h, dk, dv, BF16, ragged, start)


def test_linear_attention_prompt_then_steps():
    """A prompt in two calls, then single tokens, equals one call over all of them."""
    t, b, h, d = 150, 2, 3, 128
    q, k, v, decay, _, _ = linear_inputs(5, t, b, h, d, d, BF16, False, False)
    want, end = ref.linear(q, k, v, decay, None, None, 1.0)
    dq, dk_, dv_, dd = (x.cuda() for x in (q, k, v, decay))
    state, outs = None, []
    for lo, hi in ((0, 90), (90, 140)) + tuple((i, i + 1) for i in range(140, 150)):
        o, state = rt().linear_attention(dq[lo:hi], dk_[lo:hi], dv_[lo:hi], dd, state=state, state_out=state)
        outs.append(o)
    check_linear(torch.cat(outs).cpu().double(), state.cpu().double(), want, end, 7.0)


def test_linear_attention_ignores_what_stands_behind_the_end():
    t, b, h, d = 100, 3, 2, 64
    q, k, v, decay, state, lens = linear_inputs(9, t, b, h, d, d, BF16, True, True)
    dev = [x.cuda() for x in (q, k, v, decay)]
    one = rt().linear_attention(*dev, state=state.cuda(), lens=lens.cuda(), out=torch.zeros(v.shape, device="cuda"))
    for i in range(b):
        for x in dev[:3]:
            x[min(int(lens[i]), t):, i] = math.nan
    two = rt().linear_attention(*dev, state=state.cuda(), lens=lens.cuda(), out=torch.zeros(v.shape, device="cuda"))
    assert all(torch.equal(bits(a), bits(c)) for a, c in zip(one, two))


def test_linear_attention_large_offsets():
    """A state of more than 2^32 bytes and 2^31 elements: its ends are right."""
    b, h, d = 4104, 32, 128
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    state = torch.zeros((b, h, d, d), device="cuda")
    state[0, 0], state[-1, -1] = 1.0, 2.0
    one = torch.zeros((1, b, h, d), dtype=BF16, device="cuda")
    one[..., 0] = 1
    out, end = rt().linear_attention(one, one, one, torch.full((h,), 0.5, device="cuda"), state=state, state_out=state)
    assert end[0, 0, 0, 0] == 1.5 and end[-1, -1, 0, 0] == 2 and end[-1, -1, 127, 127] == 1
    assert end[b // 2, 3, 0, 0] == 1 and end[b // 2, 3, 1:].abs().max() == 0
    assert out[0, -1, -1, 0] == 2 and out[0, 0, 0, 5] == 0.5 and out[0, b // 2, 3, 0] == 1


# ---- 4-bit cache -----------------------------------------------------------------

def make_cache(b, hk, d, page, cols, seed, extra=3):
    """A cache whose memory is all ones (scales are NaN) and a table of scattered pages."""
    cache = rt().Kv4Cache(b * cols + extra, hk, d, page)
    cache.pool.fill_(0xFF)
    table = torch.randperm(b * cols + extra, generator=ref.gen(seed))[:b * cols].to(torch.int32).view(b, cols)
    return cache, table


def check_values(got, want):
    """value = code * scale, two float32 roundings; codes are exact."""
    off = (got.cpu().double() - want).abs()
    assert (off <= 2.0 ** -23 * want.abs()).all(), float((off / want.abs().clamp(min=1e-30)).max())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("b,hk,d,page,starts,t", [
    (1, 1, 64, 32, [0], 1),
    (3, 2, 128, 64, [0, 5, 31], 1),
    (2, 3, 128, 32, [7, 64], 70),
    (2, 1, 256, 96, [95, 0], 33),
    (4, 2, 64, 256, [0, 30, 31, 32], 2),
    (2, 5, 128, 64, [1, 63], 128),
])
def test_cache_append_read(b, hk, d, page, starts, t, dtype):
    g = ref.gen(t * 7 + d)
    cols = (max(starts) + t + page - 1) // page + 1
    cache, table = make_cache(b, hk, d, page, cols, 1)
    k, v = randn((t, b, hk, d), g, dtype), randn((t, b, hk, d), g, dtype)
    k[0, 0, 0, :64] = 0                                    # a group of zeros
    k[-1, -1, -1, 0] = 100.0
    if dtype == BF16:
        v[0, -1, 0, :64] = torch.arange(64).sub(32).to(dtype)  # largest 32: ties at 16 (3.5 steps)
    start = torch.tensor(starts, dtype=torch.int32)
    cache.append(k.cuda(), v.cuda(), table.cuda(), start.cuda())
    kr, vr = cache.read(table.cuda(), start.cuda(), t)
    check_values(kr, ref.values(k))
    check_values(vr, ref.values(v))
    # a second append behind it leaves the first as it was, and a later rewrite of part of it too
    more = randn((3, b, hk, d), g, dtype)
    cache.append(more.cuda(), more.cuda(), table.cuda(), (start + t).cuda())
    k2, v2 = cache.read(table.cuda(), start.cuda(), t)
    assert torch.equal(bits(kr), bits(k2)) and torch.equal(bits(vr), bits(v2))
    km, vm = cache.read(table.cuda(), (start + t).cuda(), 3)
    check_values(km, ref.values(more))
    check_values(vm, ref.values(more))


def test_cache_counts_holes_and_ends():
    b, hk, d, page, t = 4, 2, 128, 32, 50
    g = ref.gen(3)
    cache, table = make_cache(b, hk, d, page, 4, 2)
    table[1, 1], table[2, 0] = -1, cache.pages              # no page there
    start = torch.tensor([10, 20, 0, 100], dtype=torch.int32)   # sequence 3 runs over the table's end
    count = torch.tensor([t, 44, 40, 50], dtype=torch.int32)
    k, v = randn((t, b, hk, d), g, BF16), randn((t, b, hk, d), g, BF16)
    before = cache.pool.clone()
    cache.append(k.cuda(), v.cuda(), table.cuda(), start.cuda(), count=count.cuda())
    kr, vr = cache.read(table.cuda(), start.cuda(), t, count=count.cuda())
    p = start.long() + torch.arange(t)[:, None]
    live = torch.arange(t)[:, None] < count
    col = (p // page).clamp(max=3)
    page_of = table.long()[torch.arange(b), col]
    live &= (p < 4 * page) & (page_of >= 0) & (page_of < cache.pages)
    live = live[:, :, None, None]
    check_values(kr, torch.where(live, ref.values(k), 0.0))
    check_values(vr, torch.where(live, ref.values(v), 0.0))
    # pages that no table names, and negative starts, stay untouched
    tile = 36 * d
    used = sorted(int(x) for x in table.flatten() if 0 <= x < cache.pages)
    rest = [i for i in range(cache.pages) if i not in used]
    size = cache.nbytes // cache.pages
    for i in rest:
        assert torch.equal(cache.pool[i * size:(i + 1) * size], before[i * size:(i + 1) * size])
    assert size == hk * tile
    now = cache.pool.clone()
    cache.append(k.cuda(), v.cuda(), table.cuda(), torch.full((b,), -100, dtype=torch.int32).cuda())
    cache.append(k.cuda(), v.cuda(), table.cuda(), torch.full((b,), 2 ** 31 - 1, dtype=torch.int32).cuda())
    cache.append(k.cuda(), v.cuda(), table.cuda(), start.cuda(), count=torch.zeros(b, dtype=torch.int32).cuda())
    assert torch.equal(now, cache.pool)
    kr, _ = cache.read(table.cuda(), torch.full((b,), -20, dtype=torch.int32).cuda(), 20)
    assert (kr == 0).all()


def check_attention(got, want, mass, reach, dtype, d, sentinel):
    """Per element.  A score is a float32 sum over d channels, off by at most
    (d + 8) u of its terms' sum (reach); numerator and denominator take that
    error once each, exp2 and the sums over positions another 64 u.  bf16
    calls round each probability (half a step, relative) and the result."""
    live = ~torch.isnan(want)
    assert (got[~live] == sentinel).all()
    bound = ((2 * (d + 8) * reach + 64) * ref.U32 + (2.0 ** -8 if dtype == BF16 else 0)) * mass
    bound = bound + ref.HALF_STEP[dtype] * want.abs() * 1.001
    off = torch.where(live, (got - want).abs(), 0.0)
    bound = torch.where(live, bound, 1.0)
    assert (off <= bound).all(), float((off / bound.clamp(min=1e-30)).max())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("b,hk,group,t,n,d,page,window,sinks,holes", [
    (1, 1, 1, 1, 1, 64, 32, 0, 0, False),
    (3, 2, 4, 1, 77, 128, 32, 0, 0, False),
    (2, 1, 8, 1, 300, 128, 64, 0, 0, True),
    (2, 2, 3, 5, 130, 64, 64, 0, 0, False),
    (2, 1, 7, 2, 200, 256, 96, 50, 0, False),
    (3, 1, 2, 40, 100, 128, 32, 33, 4, True),
    (2, 1, 1, 64, 64, 64, 64, 0, 0, False),
    (2, 2, 4, 19, 260, 128, 64, 40, 70, False),
    (1, 1, 16, 3, 515, 128, 128, 1, 1, False),
    (1, 1, 20, 1, 257, 64, 32, 0, 0, False),
    (2, 1, 5, 70, 90, 256, 32, 0, 0, True),
    (1, 2, 1, 130, 400, 64, 64, 64, 2, False),
])
def test_cache_attention(b, hk, group, t, n, d, page, window, sinks, holes, dtype):
    g = ref.gen(n + t)
    cols = (n + page - 1) // page + 1
    cache, table = make_cache(b, hk, d, page, cols, n)
    k, v = randn((n, b, hk, d), g, BF16), randn((n, b, hk, d), g, BF16)
    cache.append(k.cuda(), v.cuda(), table.cuda(), torch.zeros(b, dtype=torch.int32).cuda())
    seen = torch.ones((b, n), dtype=torch.bool)
    if holes:
        table[-1, 0] = -1
        seen[-1, :page] = False
        if cols > 2:
            table[0, 1] = cache.pages + 7
            seen[0, page:2 * page] = False
    lens = torch.randint(max(1, n // 3), n + 1, (b,), generator=g, dtype=torch.int32)
    lens[0] = n
    count = None
    if b > 1:
        lens[1] = min(n, max(1, t - 1))       # fewer tokens than queries: the first queries see nothing
    if b > 2:
        lens[2] = 0
        count = torch.tensor([t, max(0, t - 2), 1], dtype=torch.int32)
    q = (2 * randn((t, b, hk * group, d), g)).to(dtype)
    scale = d ** -0.5
    kk, vv = ref.values(k).permute(1, 0, 2, 3), ref.values(v).permute(1, 0, 2, 3)
    want, mass, reach = ref.attention(q, kk, vv, seen, scale, window, sinks, lens, count)
    out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    got = cache.attention(q.cuda(), table.cuda(), lens.cuda(), dev(count), scale, window, sinks, out)
    assert got is out
    check_attention(got.cpu().double(), want, mass, reach, dtype, d, 7.0)
    again = cache.attention(q.cuda(), table.cuda(), lens.cuda(), dev(count), scale, window, sinks,
                            torch.full_like(out, 7.0))
    assert torch.equal(bits(again), bits(got))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("b,hk,group,t,n,d,page,window,sinks,holes", [
    (3, 2, 5, 4, 300, 256, 64, 0, 0, True),            # two row tiles of wide heads
    (2, 1, 8, 4, 500, 256, 32, 45, 10, True),
    (2, 2, 3, 11, 420, 256, 128, 30, 0, False),        # more
    (2, 1, 4, 90, 700, 256, 32, 100, 40, True),
    (1, 1, 2, 1, 3000, 256, 32, 0, 0, False),          # split over the cache
    (1, 1, 3, 25, 1200, 256, 32, 0, 0, True),
    (2, 1, 1, 2, 2500, 128, 32, 100, 5, False),        # windows far shorter than the cache
    (1, 2, 4, 100, 1500, 128, 64, 200, 0, False),
    (1, 1, 8, 1, 2600, 64, 32, 64, 64, True),
    (2, 1, 5, 9, 2100, 256, 96, 333, 1, False),
])
def test_cache_attention_wide_heads_and_long_caches(b, hk, group, t, n, d, page, window, sinks, holes, dtype):
    test_cache_attention(b, hk, group, t, n, d, page, window, sinks, holes, dtype)


@pytest.mark.parametrize("b,hk,group,t,n,d,page,window,sinks,holes,dtype", [
    (2, 4, 4, 300, 5600, 128, 64, 0, 0, True, BF16),   # long lists of tiles: 32 rows a wave, several parts
    (2, 4, 4, 1000, 2500, 64, 64, 1500, 40, False, BF16),
    (1, 2, 8, 260, 2600, 256, 32, 0, 0, True, BF16),
    (1, 2, 8, 130, 1500, 64, 32, 0, 0, False, F32),
])
def test_cache_attention_of_long_blocks(b, hk, group, t, n, d, page, window, sinks, holes, dtype):
    test_cache_attention(b, hk, group, t, n, d, page, window, sinks, holes, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_cache_attention_of_large_scores(dtype):
    """Scores far apart (a softmax of one), and all equal."""
    b, hk, d, page, n = 1, 1, 64, 32, 100
    cache, table = make_cache(b, hk, d, page, 4, 8)
    k, v = torch.zeros((n, b, hk, d)), randn((n, b, hk, d), ref.gen(4))
    k[37] = 100.0
    zero = torch.zeros(1, dtype=torch.int32).cuda()
    cache.append(k.to(BF16).cuda(), v.to(BF16).cuda(), table.cuda(), zero)
    q = torch.full((1, b, 2, d), 50.0, dtype=dtype)
    q[0, 0, 1] = 0
    lens = torch.tensor([n], dtype=torch.int32)
    got = cache.attention(q.cuda(), table.cuda(), lens.cuda(), scale=1.0).cpu().double()
    vv = ref.values(v.to(BF16))[:, 0, 0]
    assert torch.allclose(got[0, 0, 0], vv[37], rtol=2 ** -7, atol=0)
    # equal probabilities: their common rounding and the sum's, then the result's
    assert torch.allclose(got[0, 0, 1], vv.mean(0), rtol=2 ** -8, atol=float(vv.abs().mean()) * 2 ** -8 + 1e-6)


def test_cache_shared_pages_and_repeated_pages():
    """Two sequences that read the same pages agree; a page named twice counts twice."""
    hk, d, page = 2, 128, 32
    g = ref.gen(6)
    cache = rt().Kv4Cache(4, hk, d, page)
    k, v = randn((64, 1, hk, d), g, BF16), randn((64, 1, hk, d), g, BF16)
    cache.append(k.cuda(), v.cuda(), torch.tensor([[2, 0]], dtype=torch.int32).cuda(),
                 torch.zeros(1, dtype=torch.int32).cuda())
    q = randn((1, 1, 4, d), g, BF16).repeat(1, 2, 1, 1)
    table = torch.tensor([[2, 0], [2, 2]], dtype=torch.int32)
    lens = torch.tensor([64, 64], dtype=torch.int32)
    got = cache.attention(q.cuda(), table.cuda(), lens.cuda())
    one = cache.attention(q[:, :1].contiguous().cuda(), table[:1].cuda(), lens[:1].cuda())
    half = cache.attention(q[:, :1].contiguous().cuda(), table[:1].cuda(), lens[:1].cuda() // 2)
    assert torch.allclose(got[:, :1].float(), one.float(), rtol=2 ** -6, atol=2 ** -7)
    assert torch.allclose(got[:, 1:].float(), half.float(), rtol=2 ** -6, atol=2 ** -7)


def test_cache_of_more_than_4_gib():
    hk, d, page = 1, 128, 64
    pages = (5 << 30) // (page * 144)
    cache = rt().Kv4Cache(pages, hk, d, page)
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32)
    g = ref.gen(12)
    k, v = randn((150, 1, hk, d), g, BF16), randn((150, 1, hk, d), g, BF16)
    zero = torch.zeros(1, dtype=torch.int32).cuda()
    cache.append(k.cuda(), v.cuda(), table.cuda(), zero)
    kr, vr = cache.read(table.cuda(), zero, 150)
    check_values(kr, ref.values(k))
    check_values(vr, ref.values(v))
    q = randn((1, 1, 4, d), g, BF16)
    lens = torch.tensor([150], dtype=torch.int32)
    kk, vv = ref.values(k).permute(1, 0, 2, 3), ref.values(v).permute(1, 0, 2, 3)
    want, mass, reach = ref.attention(q, kk, vv, torch.ones((1, 150), dtype=torch.bool), d ** -0.5, 0, 0, lens, None)
    got = cache.attention(q.cuda(), table.cuda(), lens.cuda())
    check_attention(got.cpu().double(), want, mass, reach, BF16, d, 7.0)


# ---- as they are used ----------------------------------------------------------

def layer_step(cache, table, lens, rows, weights, pos, freq, state, decay, bufs):
    """One decode step of a softmax layer and a linear layer: packed projections in, both outputs."""
    hq, hk, d = 8, 2, 128
    n = rows.shape[0]
    q, k = rt().qk_norm_rope(rows[:, :hq * d].view(n, hq, d), rows[:, hq * d:(hq + hk) * d].view(n, hk, d), "rms",
                             *weights, pos=pos, inv_freq=freq, q_out=bufs["q"], k_out=bufs["k"])
    v = rows[:, (hq + hk) * d:].view(1, n, hk, d)
    bufs["v"].copy_(v)
    cache.append(k.view(1, n, hk, d), bufs["v"], table, pos)
    o = cache.attention(q.view(1, n, hq, d), table, lens, out=bufs["o"], workspace=bufs["ws"])
    lo, _ = rt().linear_attention(q.view(1, n, hq, d), q.view(1, n, hq, d), o, decay, state=state, state_out=state,
                                  out=bufs["lo"])
    return o, lo


def test_layers_together_eager_stream_and_graph():
    """Norms, cache and both attentions in a row: the same on another stream, and in a graph that is
    replayed with the program's own work between, each replay against the eager step."""
    hq, hk, d, b, page = 8, 2, 128, 3, 32
    g = ref.gen(21)
    weights = ((1 + 0.1 * randn((d,), g)).cuda(), (1 + 0.1 * randn((d,), g)).cuda())
    freq = torch.exp(-torch.arange(32) / 4.0).float().cuda()
    decay = torch.linspace(0.5, 1.0, hq).cuda()
    steps = [randn((b, (hq + 2 * hk) * d), g, BF16).cuda() for _ in range(6)]
    table = torch.randperm(3 * b, generator=g).to(torch.int32).view(b, 3).cuda()
    first = torch.tensor([0, 30, 63], dtype=torch.int32).cuda()

    def fresh():
        cache = rt().Kv4Cache(3 * b, hk, d, page)
        cache.pool.zero_()
        gk = ref.gen(22)
        past = randn((64, b, hk, d), gk, BF16).cuda()
        cache.append(past, past, table, torch.zeros_like(first), count=first)
        bufs = dict(q=torch.empty((b, hq, d), dtype=BF16, device="cuda"), k=torch.empty((b, hk, d), dtype=BF16, device="cuda"),
                    v=torch.empty((1, b, hk, d), dtype=BF16, device="cuda"), o=torch.empty((1, b, hq, d), dtype=BF16, device="cuda"),
                    lo=torch.empty((1, b, hq, d), device="cuda"))
        bufs["ws"] = cache.attention_workspace(bufs["o"], table)
        return cache, bufs, torch.zeros((b, hq, d, d), device="cuda")

    def eager():
        cache, bufs, state = fresh()
        got = []
        for i, rows in enumerate(steps):
            o, lo = layer_step(cache, table, first + i + 1, rows, weights, first + i, freq, state, decay, bufs)
            got.append((o.clone(), lo.clone()))
        return got, state, cache

    want, state_w, cache_w = eager()
    assert all(torch.isfinite(x.float()).all() for pair in want for x in pair)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, state_g, cache_g = eager()
    side.synchronize()
    for a, c in zip(want, got):
        assert all(torch.equal(bits(x), bits(y)) for x, y in zip(a, c))
    assert torch.equal(cache_w.pool, cache_g.pool) and torch.equal(bits(state_w), bits(state_g))

    cache, bufs, state = fresh()
    rows, pos, lens = torch.empty_like(steps[0]), torch.empty_like(first), torch.empty_like(first)
    rows.copy_(steps[0]), pos.copy_(first), lens.copy_(first + 1)
    keep, keep_pool = state.clone(), cache.pool.clone()
    with torch.cuda.stream(side):       # warm-up outside of the capture
        layer_step(cache, table, lens, rows, weights, pos, freq, state, decay, bufs)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o, lo = layer_step(cache, table, lens, rows, weights, pos, freq, state, decay, bufs)
    state.copy_(keep), cache.pool.copy_(keep_pool)
    for i in range(len(steps)):
        rows.copy_(steps[i]), pos.copy_(first + i), lens.copy_(first + i + 1)
        graph.replay()
        assert torch.equal(bits(o), bits(want[i][0])) and torch.equal(bits(lo), bits(want[i][1])), i
        torch.cuda.synchronize()
    assert torch.equal(bits(state), bits(state_w)) and torch.equal(cache.pool, cache_w.pool)


def test_norm_feeds_the_gated_delta_rule():
    """L2 norms of raw projections in front of pace_decode_period: the library's own q, k to bf16 rounding."""
    import numpy as np

    from linear_attn_decode_pace_amd import inputs, pace
    runtime = rt()
    w = inputs.ragged("norm-feed", 77, B=3, H=4, n_int8=1, steps=8)
    tok = runtime.DeviceTokens(inputs.tokens(w, 0, inputs.SEG_DECODE, 0, 8))
    raw_q, raw_k = (tok.q.float() * 5).to(BF16), (tok.k.float() * 0.25).to(BF16)
    q, k = runtime.qk_norm_rope(raw_q.view(-1, w.H, w.dk), raw_k.view(-1, w.H, w.dk), "l2", eps=0.0)
    outs = []
    for a, c in ((tok.q, tok.k), (q.view_as(tok.q), k.view_as(tok.k))):
        st = runtime.State(w, inputs.head_bits(w, 0), pace.PACE_INIT_F32, runtime.warmup_state(w, 0))
        tok.q, tok.k = a, c
        out = runtime.out_buffer(w, 8)
        st.decode(tok, out)
        outs.append(out.double().cpu().numpy())
        st.free()
    # q and k differ by the bf16 roundings of the detour (two of 2^-9 each, in both); o is linear in q and
    # quadratic in k at most
    off = np.linalg.norm(outs[0] - outs[1]) / np.linalg.norm(outs[0])
    assert off < 6 * 2.0 ** -8, off


def test_wrapper_refusals():
    r = rt()
    x = torch.zeros((4, 2, 64), device="cuda")
    with pytest.raises(TypeError):
        r.qk_norm_rope(x.half())
    with pytest.raises(TypeError):
        r.qk_norm_rope(x, x.to(BF16))
    with pytest.raises(ValueError):
        r.qk_norm_rope(x, norm="batch")
    with pytest.raises(ValueError):
        r.qk_norm_rope(x[:, :, ::2])
    with pytest.raises(ValueError):
        r.qk_norm_rope(x.transpose(0, 1))
    with pytest.raises(ValueError):
        r.qk_norm_rope(x, x[:3])
    with pytest.raises(ValueError):
        r.qk_norm_rope(x[:1].expand(4, 2, 64))                  # rows overlap
    with pytest.raises(TypeError):
        r.qk_norm_rope(x, inv_freq=torch.ones(4, device="cuda"), pos=torch.zeros(4, device="cuda"))
    with pytest.raises(TypeError):
        r.qk_norm_rope(x, inv_freq=torch.ones(4, device="cuda"))
    with pytest.raises(r.pace.PaceError):
        r.qk_norm_rope(x, inv_freq=torch.ones(33, device="cuda"), pos=torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        r.qk_norm_rope(x, q_out=torch.empty((4, 2, 64)))
    with pytest.raises(TypeError):
        r.qk_norm_rope(x, stream=0)
    y = torch.zeros((3, 2, 2, 64), dtype=BF16, device="cuda")
    d = torch.ones(2, device="cuda")
    with pytest.raises(ValueError):
        r.linear_attention(y, y, y, d[:1])
    with pytest.raises(ValueError):
        r.linear_attention(y, y[:2], y, d)
    with pytest.raises(ValueError):
        r.linear_attention(y.transpose(1, 2), y, y, d)
    with pytest.raises(TypeError):
        r.linear_attention(y, y, y, d, lens=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        r.linear_attention(y, y, y, d, lens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        r.linear_attention(y, y, y, d, state=torch.zeros((2, 2, 64, 64), dtype=BF16, device="cuda"))
    with pytest.raises(r.pace.PaceError):
        r.linear_attention(y, y, y[..., :24].contiguous(), d)
    cache = r.Kv4Cache(4, 2, 64, 32)
    table, n = torch.zeros((2, 2), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        cache.append(y[..., :32].contiguous(), y[..., :32].contiguous(), table, n)
    with pytest.raises(TypeError):
        cache.append(y, y.float(), table, n)
    with pytest.raises(TypeError):
        cache.append(y, y, table.long(), n)
    with pytest.raises(ValueError):
        cache.append(y, y, table[:1], n)
    with pytest.raises(ValueError):
        cache.read(table, n, 0)
    with pytest.raises(r.pace.PaceError):
        cache.attention(y.repeat(1, 1, 2, 1)[:, :, :3].contiguous(), table, n)   # 3 query heads on 2
    with pytest.raises(r.pace.PaceError):
        cache.attention(y, table, n, window=-1)
    with pytest.raises(TypeError):
        cache.attention(y, table, n, workspace=torch.empty(1 << 20, device="cuda")) \
            if cache.attention_workspace(y, table) is not None else cache.attention(y, table, n, stream=1)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_cache_codes_are_exact(dtype):
    """Every pair of a bf16 mantissa and a group's largest value, far apart in size too: codes are those of
    the exact quotient (its ties are exact in float32), scales within a rounding."""
    d, page = 64, 32
    tops = torch.cat([torch.arange(128, 256) * 2.0 ** e for e in (-7, 3, -120, 113)])
    n = tops.numel() * 4
    g = ref.gen(31)
    x = torch.zeros((n, 1, 1, d))
    for i in range(n):
        top = tops[i % tops.numel()]
        m = torch.randint(128, 256, (d,), generator=g) * 2.0 ** torch.randint(-4, 1, (d,), generator=g)
        v = (m / 255 * top).to(BF16).float() * torch.where(torch.rand(d, generator=g) < 0.5, -1.0, 1.0)
        v = torch.where(v.abs() > top, top, v)
        v[i % d] = top
        if i % 3 == 0:
            v[(i + 1) % d] = -top / 2           # a tie: 3.5 steps
        x[i, 0, 0] = v
    x = x.to(dtype)
    cache, table = make_cache(1, 1, d, page, (n + page - 1) // page, 5)
    zero = torch.zeros(1, dtype=torch.int32).cuda()
    cache.append(x.cuda(), x.cuda(), table.cuda(), zero)
    for got in cache.read(table.cuda(), zero, n):
        check_values(got, ref.values(x))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-38])
def test_cache_attention_of_unusual_scales(scale, dtype):
    b, hk, group, t, n, d, page = 2, 2, 3, 7, 150, 128, 64
    g = ref.gen(17)
    cache, table = make_cache(b, hk, d, page, 3, 4)
    k, v = randn((n, b, hk, d), g, BF16), randn((n, b, hk, d), g, BF16)
    cache.append(k.cuda(), v.cuda(), table.cuda(), torch.zeros(b, dtype=torch.int32).cuda())
    q = randn((t, b, hk * group, d), g, dtype)
    lens = torch.tensor([n, 40], dtype=torch.int32)
    kk, vv = ref.values(k).permute(1, 0, 2, 3), ref.values(v).permute(1, 0, 2, 3)
    want, mass, reach = ref.attention(q, kk, vv, torch.ones((b, n), dtype=torch.bool), scale, 0, 0, lens, None)
    got = cache.attention(q.cuda(), table.cuda(), lens.cuda(), scale=scale)
    check_attention(got.cpu().double(), want, mass, reach, dtype, d, 7.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_cache_of_the_largest_and_smallest_values(dtype):
    """Groups near the largest finite value and of the smallest normal ones.  Scales of the latter are
    denormal: half a step of 2^-149 for each of up to 7 steps."""
    d, page, n = 64, 32, 8
    g = ref.gen(19)
    x = randn((n, 1, 1, d), g)
    x = x / x.abs().amax(-1, keepdim=True)
    size = torch.tensor([3.3e38, 1e38, 3e37, 1e30, 1e-30, 1e-37, 1.2e-38, 1.0])
    x = (x * size[:, None, None, None]).to(dtype)
    assert torch.isfinite(x.float()).all()
    cache, table = make_cache(1, 1, d, page, 1, 5)
    zero = torch.zeros(1, dtype=torch.int32).cuda()
    cache.append(x.cuda(), x.cuda(), table.cuda(), zero)
    want = ref.values(x)
    for got in cache.read(table.cuda(), zero, n):
        off = (got.cpu().double() - want).abs()
        assert (off <= 2.0 ** -23 * want.abs() + 7 * 2.0 ** -149).all()


def test_norm_of_keys_alone():
    """heads_q = 0 through the C entry point."""
    from linear_attn_decode_pace_amd import pace
    g = ref.gen(23)
    k = randn((5, 3, 128), g, BF16)
    out = torch.empty((5, 3, 128), dtype=BF16, device="cuda")
    cfg = pace.pace_norm_config(5, 0, 3, 128, pace.PACE_DTYPE_BF16, pace.PACE_NORM_L2, 1e-6, 9.0, 0, 0, 0, 3 * 128)
    pace.pace_qk_norm_rope(cfg, None, k.cuda(), None, None, None, None, None, out)
    y = ref.norm_rope(k, "l2", None, 1e-6, None, None, False, 1.0)
    assert ((out.cpu().double() - y).abs() <= norm_bound(y, BF16, 128)).all()


def test_two_calls_at_once():
    """Calls on two streams with buffers of their own equal the same calls one after another."""
    g = ref.gen(29)
    q, k, v, decay, state, _ = linear_inputs(40, 1500, 2, 4, 128, 128, BF16, False, True)
    one = [x.cuda() for x in (q, k, v, decay, state)]
    two = [x.cuda() for x in (k, q, v, decay, state * 2)]
    cache, table = make_cache(4, 2, 128, 64, 40, 3)
    kk, vv = randn((2500, 4, 2, 128), g, BF16).cuda(), randn((2500, 4, 2, 128), g, BF16).cuda()
    cache.append(kk, vv, table.cuda(), torch.zeros(4, dtype=torch.int32).cuda())
    qa, lens = randn((3, 4, 8, 128), g, BF16).cuda(), torch.tensor([2500, 100, 1999, 2048], dtype=torch.int32).cuda()
    table = table.cuda()

    def calls(x, s):
        o, e = rt().linear_attention(*x[:4], state=x[4], stream=s)
        return o, e, cache.attention(qa, table, lens, stream=s)

    want = calls(one, None), calls(two, None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [calls(x, s) for x, s in zip((one, two), streams)]
    torch.cuda.synchronize()
    for a, c in zip(want, got):
        assert all(torch.equal(bits(x), bits(y)) for x, y in zip(a, c))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_cache_channels_of_zeros_stay_zero(dtype):
    """Value channels that are zero in every token give exactly zero."""
    b, hk, d, page, n = 2, 2, 128, 64, 700
    g = ref.gen(37)
    cache, table = make_cache(b, hk, d, page, 11, 6)
    k, v = randn((n, b, hk, d), g, BF16), randn((n, b, hk, d), g, BF16)
    v[..., 5], v[..., 64:] = 0, 0
    cache.append(k.cuda(), v.cuda(), table.cuda(), torch.zeros(b, dtype=torch.int32).cuda())
    lens = torch.tensor([n, 3], dtype=torch.int32).cuda()
    for t in (1, 30):                  # both kernels
        q = randn((t, b, hk * 4, d), g, dtype).cuda()
        got = cache.attention(q, table.cuda(), lens)
        assert (got[..., 5] == 0).all() and (got[..., 64:] == 0).all() and (got[-1, ..., :5] != 0).any()
