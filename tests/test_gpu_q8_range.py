"""The attention over the quantised cache where softmax weights span a wide
range: long contexts under one large weight, rows of zeros, scales of any
kind.  Compared with the definition in 64 bits; caches come from
ic_cache_write_q8 unless a test makes its own.

Tolerance, elementwise, with softmax weights p_s (normalised), scales g_s,
codes c_s, V_s = g_s c_s and w_s = p_s g_s.  Nothing in it is a bias that adds
up over positions:

    2^-8 |ref|            the output's rounding to bfloat16
  + 2^-7 sum_s p_s |V_s|  a weight is an e4m3 number and an e5m2 number for the
                          rest.  The first is off by at most 2^-4 of the
                          weight's power of two 2^E, so the rest is at most
                          2^(E-4), where e5m2 steps are at most 2^(E-7): the
                          whole step, since weights may be rounded up or down
                          at random
  + 4 sqrt(sum_s (t_s |c_s|)^2)
                          smaller weights, t_s the step of e5m2 there.  With the
                          row's largest weight at 2^4 (it stands there or
                          higher), weights under 2^-6 leave a rest of 2^-10 at
                          most, step 2^-13; under 2^-10 the rest is the weight,
                          its step a quarter of it at most, and never under
                          2^-16: t = max(min(2^-13, w / 4), 2^-16) for w <
                          2^-6.  They are rounded at random, by independent
                          errors of mean 0 in intervals of length t: by
                          Hoeffding's inequality the sum exceeds 4 sqrt(sum
                          t^2) with probability under 2 exp(-32) = 3e-14
  + sum_s t_s |c_s| / 2   over the small weights that share an aligned group of
                          four entries with one of 2^1 or more (2^-7.5 of the
                          largest at least, which may have grown to 2^8.5):
                          these are rounded to the nearest
  + 2 d sum_s p_s |V_s|   the logits' error d: float32 sums of 576 products,
                          each 2^-24 of the sum of absolute terms; q kept to
                          2^-17 of its row's largest value; 2^-21 of the logit,
                          2^-21 for exp, 2^-17 for the base-2 logarithm of a
                          scale that is no power of two (a float32 number up to
                          128, half a step 2^-18, once in itself and once in
                          the sum with the logit).  A weight is off by d and so
                          is the normaliser

A row of zeros among the values has no part in O; its weight stands for 2^-40
p_s when the largest weight is sought.
"""
import numpy as np
import pytest
import torch

import cross_layer_top_full_b200 as ic
from parity_util import check_attention

pytestmark = pytest.mark.gpu
BF, D = torch.bfloat16, "cuda:0"
LN2 = float(np.log(2.0))


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ic.lib()


def new_ws(nbytes=256):
    ws = torch.empty(max(nbytes, ic.STATUS_BYTES), dtype=torch.uint8, device=D)
    ic.workspace_init(ws)
    return ws


def packed(kv):
    """Cache rows and scales of latent rows [n, 576], by the library's writer; n is padded to whole pages of 128."""
    n = len(kv)
    rows = -(-n // 128) * 128
    cache = torch.zeros(rows, 640, dtype=torch.uint8, device=D)
    scale = torch.ones(rows, device=D)
    ws = new_ws()
    ic.cache_write_q8(torch.arange(n, dtype=torch.int32, device=D), ws, kv=kv.float(), kv_q8=cache, kv_scale=scale)
    assert ic.read_status(ws) == 0
    return cache, scale


def attend(q, cache, scale, lens, idx=None, tree=None, factor=576 ** -0.5, status=0):
    """q [B, Lq, Hq, 576]; every sequence reads the same pages 0, 1, .. of the cache."""
    B, Lq, Hq, _ = q.shape
    T = max(lens)
    pages = -(-T // 128)
    table = torch.arange(pages, dtype=torch.int32, device=D).repeat(B, 1)
    d_lens = torch.tensor(lens, dtype=torch.int32, device=D)
    pr = ic.paged_rows(d_lens, table, T, 128, len(cache) // 128, Lq)
    ws = new_ws(ic.tree_attn_q8_workspace_size(pr, 0 if idx is None else idx.shape[-1], Hq))
    out = torch.full((B, Lq, Hq, 512), 3.0, dtype=BF, device=D)
    ic.tree_attn_q8_paged(q, cache, scale, idx, pr, factor, out, ws, tree=tree)
    assert ic.read_status(ws) == status
    return out


def exact(q, cache, scale, at, factor, group=None):
    """Heads q [H, 576] over cache rows `at` (list order): the output and its tolerance, float64."""
    codes = cache[at, :512].view(torch.float8_e4m3fn).double()
    g = scale[at].double()
    k = torch.cat([codes, cache[at, 512:].view(BF).double()], 1) * g[:, None]
    q = q.double()
    s = q @ k.T * factor
    p = torch.softmax(s, 1)
    ref = p @ k[:, :512]
    nil = (codes == 0).all(1)
    w = torch.where(nil, p * 2.0 ** -40, p * g)
    u = w / w.amax(1, keepdim=True) * 16.0                               # the largest at 2^4
    t = torch.where(u < 2.0 ** -6, torch.clamp(torch.clamp(u / 4, max=2.0 ** -13), min=2.0 ** -16), 0.0)
    t = torch.where(nil, 0.0, t)
    entry = torch.arange(len(at), device=D) if group is None else group
    four = entry // 4
    big = torch.zeros(len(q), int(four.max()) + 1, dtype=torch.float64, device=D)
    big.scatter_reduce_(1, four.expand_as(u), u, "amax")
    near = t * (big[:, four] >= 2.0 ** -3.5)
    unit = w.amax(1, keepdim=True) / 16.0
    c = codes.abs()
    v = p @ k[:, :512].abs()
    terms = q.abs() @ k.abs().T * abs(factor)
    floor = q.abs().amax(1, keepdim=True) * k.abs().sum(1) * abs(factor)
    d = (576 * 2.0 ** -24 * terms + 2.0 ** -17 * floor + 2.0 ** -21 * s.abs() + 2.0 ** -21 + 2.0 ** -17).amax(1)
    tol = (2.0 ** -8 * ref.abs() + 2.0 ** -7 * v + unit * (4 * ((t * t) @ (c * c)).sqrt() + near @ c / 2)
           + 2 * d[:, None] * v)
    return ref, tol


def check(got, ref, tol, what):
    assert torch.isfinite(got.float()).all(), what
    over = ((got.double() - ref).abs() / (tol + 1e-300)).max()
    assert over <= 1, "%s: %.3f of the tolerance" % (what, float(over))


def one_above(n, bits, first, spread=0.0, seed=1):
    """n positions whose logits (through columns that carry no value) lie `bits` powers of two under position 0's,
    scattered by a normal distribution of `spread` nats; values of size 1 that do not cancel."""
    g = torch.Generator(device=D).manual_seed(seed)
    kv = torch.zeros(n, 576, device=D)
    kv[:, :512] = 1.0 + 0.25 * torch.sin(torch.arange(n, device=D)[:, None] * 0.7 + torch.arange(512, device=D))
    kv[0, :512] = first
    kv[0, 512:544] = bits * LN2
    if spread:
        kv[1:, 544:576] = spread * torch.randn(n - 1, 1, device=D, generator=g)
    q = torch.zeros(576, device=D)
    q[512:] = 1.0 / 32
    return kv, q.to(BF)


# ---------------------------------------------------------------- small weights over long contexts
@pytest.mark.parametrize("n,bits,spread", [
    (65536, 17.0, 0.0), (65536, 17.4, 0.0), (65536, 18.5, 0.0), (65536, 19.1, 0.0), (65536, 20.0, 0.0),
    (65536, 14 / LN2, 1.0), (200000, 14 / LN2, 1.0), (200000, 19.5, 0.0), (8192, 17.4, 0.0), (8192, 13.3, 0.0),
])
def test_small_weights_of_a_long_context_count(n, bits, spread):
    """64 nodes of 128 heads read one sequence: a unit's positions stay together, under one maximum."""
    Lq = 64
    kv, q = one_above(n, bits, -1.0, spread)
    cache, scale = packed(kv)
    mask = torch.full((1, Lq), -1, dtype=torch.int64, device=D)          # every row sees every position
    out = attend(q.expand(1, Lq, 128, 576).contiguous(), cache, scale, [n], tree=mask, factor=1.0)
    ref, tol = exact(q[None], cache, scale, torch.arange(n, device=D), 1.0)
    for i in (0, 7, 31, 63):
        check(out[0, i], ref, tol, "node %d" % i)
    rows = out[0].reshape(-1, 512)
    check_attention(rows[None].double().cpu().numpy(), ref.expand(len(rows), 512)[None].cpu().numpy(), "every row")


@pytest.mark.parametrize("bits,first", [(13.0, -1.0), (16.0, 0.0), (18.5, 0.0), (19.1, 3.0)])
def test_small_weights_of_long_lists_count(bits, first):
    """128 lists of 16384 positions each, in several orders; position 0 is in all of them."""
    n, k, B, Lq = 40000, 16384, 8, 16
    kv, q = one_above(n, bits, first)
    cache, scale = packed(kv)
    g = torch.Generator(device=D).manual_seed(3)
    idx = torch.stack([torch.randperm(n - Lq - 1, device=D, generator=g)[:k] + 1 for _ in range(B * Lq)])
    idx[torch.arange(B * Lq), torch.randint(0, k, (B * Lq,), device=D, generator=g)] = 0
    idx = idx.view(B, Lq, k).to(torch.int32)
    out = attend(q.expand(B, Lq, 128, 576).contiguous(), cache, scale, [n] * B, idx=idx, factor=1.0)
    for b, i in ((0, 0), (3, 9), (7, 15)):
        ref, tol = exact(q[None], cache, scale, idx[b, i].long(), 1.0)
        check(out[b, i], ref, tol, "list %d %d" % (b, i))
        check_attention(out[b, i][None].double().cpu().numpy(), ref.expand(128, 512)[None].cpu().numpy(), "list")


def test_unlike_small_weights_beside_a_large_one():
    """Every fourth of the small weights is a thousand times the others: each kind keeps its share."""
    n, Lq = 65536, 64
    kv, q = one_above(n, 9.0, 0.0)
    kv[:, 544:576] = torch.where(torch.arange(n, device=D) % 4 == 1, 0.0, -10 * LN2)[:, None]
    kv[:, :512] = torch.where((torch.arange(n, device=D) % 4 == 1)[:, None], kv[:, :512] / 1024, kv[:, :512])
    cache, scale = packed(kv)
    mask = torch.full((1, Lq), -1, dtype=torch.int64, device=D)
    out = attend(q.expand(1, Lq, 128, 576).contiguous(), cache, scale, [n], tree=mask, factor=1.0)
    ref, tol = exact(q[None], cache, scale, torch.arange(n, device=D), 1.0)
    check(out[0].reshape(-1, 512), ref, tol, "every row")


# ---------------------------------------------------------------- rows of zeros
@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("size,below", [(1.0, 0.0), (1.0, 8.0), (1e-2, 3.0), (2e-4, 0.0), (1e-4, 3.0), (1e-6, 1.0)])
def test_a_row_of_zeros_does_not_hide_the_others(size, below, listed):
    """Tokens whose 512 values are 0, with logits above the others', among tokens of one size."""
    n, B = 2048, 80
    g = torch.Generator(device=D).manual_seed(5)
    kv = torch.randn(n, 576, device=D, generator=g) * size
    kv[:, 512:] = 0.0
    zeros = torch.tensor([3, 700, 701, 1500, 2047], device=D)
    kv[zeros] = 0.0
    kv[zeros, 512:544] = below
    q = torch.zeros(2, 576, device=D)
    q[:, 512:] = 1.0 / 32
    q[1, :512] = torch.randn(512, device=D, generator=g) / (size * 40)
    q = q.to(BF)
    cache, scale = packed(kv)
    cache[zeros[1], 100] = 0x80                                          # -0 is a 0 too
    at = torch.arange(n, device=D)
    idx = at.to(torch.int32).expand(B, 1, n).contiguous() if listed else None
    out = attend(q.expand(B, 1, 2, 576).contiguous(), cache, scale, [n] * B, idx=idx, factor=1.0)
    ref, tol = exact(q, cache, scale, at, 1.0)
    for b in (0, 41, 79):
        check(out[b, 0], ref, tol, "sequence %d" % b)


def test_many_rows_of_zeros():
    """Whole pages of zeros, between tokens; and a sequence of nothing else gives zeros."""
    n = 1500
    g = torch.Generator(device=D).manual_seed(6)
    kv = torch.randn(n, 576, device=D, generator=g) * 1e-3
    kv[100:1200, :512] = 0.0
    q = torch.randn(1, 1, 20, 576, device=D, generator=g).to(BF)
    cache, scale = packed(kv)
    ref, tol = exact(q[0, 0], cache, scale, torch.arange(n, device=D), 576 ** -0.5)
    check(attend(q, cache, scale, [n])[0, 0], ref, tol, "pages of zeros")
    cache, scale = packed(torch.zeros(300, 576, device=D))
    assert (attend(q, cache, scale, [300]) == 0).all()


def test_a_single_value_is_no_row_of_zeros():
    """Rows of scale 1 with one value anywhere, rows of zeros beside them."""
    n = 700
    g = torch.Generator(device=D).manual_seed(11)
    kv = torch.zeros(n, 576, device=D)
    kv[::5] = torch.randn(140, 576, device=D, generator=g)
    columns = torch.arange(512, device=D)
    at = torch.arange(n, device=D)[torch.arange(n, device=D) % 5 != 0][:512]
    kv[at, columns] = 300.0 * (1 - 2 * (columns % 2))
    q = torch.zeros(1, 1, 9, 576, device=D)
    q[..., 512:] = torch.randn(1, 1, 9, 64, device=D, generator=g)
    q = q.to(BF)
    cache, scale = packed(kv)
    ref, tol = exact(q[0, 0], cache, scale, torch.arange(n, device=D), 576 ** -0.5)
    check(attend(q, cache, scale, [n])[0, 0], ref, tol, "one value a row")


# ---------------------------------------------------------------- scales
@pytest.mark.parametrize("listed", [False, True])
def test_scales_that_are_no_powers_of_two(listed):
    """A cache that was filled by another rule: absmax / 448."""
    n = 900
    g = torch.Generator(device=D).manual_seed(7)
    kv = torch.randn(n, 576, device=D, generator=g) * torch.exp(torch.randn(n, 1, device=D, generator=g))
    scale = torch.ones(1024, device=D)
    scale[:n] = kv[:, :512].abs().amax(1) / 448.0
    cache = torch.zeros(1024, 640, dtype=torch.uint8, device=D)
    cache[:n, :512] = (kv[:, :512] / scale[:n, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    cache[:n, 512:] = (kv[:, 512:] / scale[:n, None]).to(BF).view(torch.uint8).view(n, 128)
    q = torch.randn(1, 2, 70, 576, device=D, generator=g).to(BF)
    idx = None
    if listed:
        idx = torch.stack([torch.randperm(n - 2, device=D, generator=g)[:333] for _ in range(2)]).view(1, 2, 333).to(torch.int32)
    out = attend(q, cache, scale, [n], idx=idx)
    for i in range(2):
        at = torch.arange(n - 1 + i, device=D) if idx is None else idx[0, i].long()
        ref, tol = exact(q[0, i], cache, scale, at, 576 ** -0.5)
        check(out[0, i], ref, tol, "node %d" % i)


def test_large_and_small_scales():
    """One value in each row far from the others' sizes: scales 2^-32 to 2^40 in turn, one at a time."""
    g = torch.Generator(device=D).manual_seed(8)
    q = torch.randn(1, 1, 8, 576, device=D, generator=g).to(BF)
    for e in (-32, -20, 0, 25, 40):
        kv = torch.randn(200, 576, device=D, generator=g) * 2.0 ** e * 100
        kv[:, :512].clamp_(-300 * 2.0 ** e, 300 * 2.0 ** e)
        cache, scale = packed(kv)
        factor = 2.0 ** -e / 2400
        ref, tol = exact(q[0, 0], cache, scale, torch.arange(200, device=D), factor)
        check(attend(q, cache, scale, [200], factor=factor)[0, 0], ref, tol, "scale 2^%d" % e)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf"), -0.5, 0.0, 1e-40])
@pytest.mark.parametrize("listed", [False, True])
def test_a_bad_scale_stays_where_it_is_seen(bad, listed):
    """A scale that is no positive normal number makes the rows that see it NaN, and no others."""
    n, Lq, Hq = 200, 5, 20
    g = torch.Generator(device=D).manual_seed(9)
    cache, scale = packed(torch.randn(n, 576, device=D, generator=g))
    scale[196] = bad                                                     # node 1
    q = torch.randn(1, Lq, Hq, 576, device=D, generator=g).to(BF)
    masks = [1, 3, 1 | 4, 1 | 8, 1 | 2 | 16]
    tree = torch.tensor([masks], dtype=torch.int64, device=D)
    idx = torch.arange(n, dtype=torch.int32, device=D).expand(1, Lq, n).contiguous() if listed else None
    out = attend(q, cache, scale, [n], idx=idx, tree=tree)
    for i, mask in enumerate(masks):
        if mask & 2:
            assert torch.isnan(out[0, i]).all(), i
            continue
        at = torch.tensor([s for s in range(n) if s < 195 or mask >> (s - 195) & 1], device=D)
        ref, tol = exact(q[0, i], cache, scale, at, 576 ** -0.5, group=at)
        check(out[0, i], ref, tol, "node %d" % i)


@pytest.mark.parametrize("listed", [False, True])
def test_rows_that_were_never_written_are_rows_of_zeros(listed):
    """Bytes and scales of a fresh cache, all 0, among small values."""
    n = 300
    g = torch.Generator(device=D).manual_seed(10)
    cache, scale = packed(torch.randn(n, 576, device=D, generator=g) * 1e-3)
    fresh = torch.tensor([17, 250], device=D)
    cache[fresh], scale[fresh] = 0, 0.0
    ones = scale.clone()
    ones[fresh] = 1.0
    q = torch.randn(1, 3, 11, 576, device=D, generator=g).to(BF)
    idx = torch.arange(n, dtype=torch.int32, device=D).expand(1, 3, n).contiguous() if listed else None
    out = attend(q, cache, scale, [n], idx=idx)
    for i in range(3):
        ref, tol = exact(q[0, i], cache, ones, torch.arange(n - 2 + i, device=D), 576 ** -0.5)
        check(out[0, i], ref, tol, "node %d" % i)
    assert (attend(q, cache * 0, scale * 0, [n], idx=idx) == 0).all()
