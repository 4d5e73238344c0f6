"""The quantised cache on the GPU: writing, reading back and the attention of
drafted tokens, against the 64-bit numpy definition in q8_util.py.

Writing and reading are exact: codes, scales and values must be equal.  The
attention's tolerance is derived in q8_util.py."""
import numpy as np
import pytest
import torch

import cross_layer_top_full_b200 as ic
import oracle
import q8_util as u8
from parity_util import check_attention, check_topk_band, host64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
INDEX_RANGE = 1


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ic.lib()
    return torch.device("cuda:0")


def make_ws(nbytes, dev):
    ws = torch.empty(max(nbytes, ic.STATUS_BYTES), dtype=torch.uint8, device=dev)
    ic.workspace_init(ws)
    return ws


def caches(rows, dev, fill=0xA5):
    """Latent and indexer caches whose bytes show whether they were touched."""
    return dict(kv_q8=torch.full((rows, 640), fill, dtype=torch.uint8, device=dev),
                kv_scale=torch.full((rows,), -3.0, device=dev),
                k_codes=torch.full((rows, 128), fill, dtype=torch.uint8, device=dev),
                k_scale=torch.full((rows,), -3.0, device=dev))


def activations(n, width, seed, dtype, special=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, width, generator=g) * torch.exp(torch.randn(n, 1, generator=g))
    if special:
        edge = [0.0, -0.0, float("inf"), float("-inf"), float("nan"), 1e-30, -3e38, 448.0, 225.0,
                2.0 ** -133, 17.0, 19.0, 1.0625, 0.03125 * 1.5]
        for r in range(n):
            if r % 7 == 0:
                x[r] = 0.0                                    # a row of zeros
            elif r % 7 == 1:
                x[r, r % width] = 448.0 * 2.0 ** (r % 11 - 5)  # at a scale's border
                x[r].clamp_(-448.0 * 2.0 ** (r % 11 - 5), 448.0 * 2.0 ** (r % 11 - 5))
            elif r % 7 == 2:
                for i, v in enumerate(edge):
                    x[r, (37 * i + r) % width] = v
            elif r % 7 == 3:
                x[r] *= 1e-12
            elif r % 7 == 4:
                x[r] = float("nan")
    return x.to(dtype)


def wide(x, extra, offset, dev):
    """x on the device as a view of wider rows, starting `offset` elements in."""
    big = torch.full((x.shape[0], x.shape[1] + extra), 7.0, dtype=x.dtype, device=dev)
    view = big[:, offset:offset + x.shape[1]]
    view.copy_(x)
    return view


def num(x):
    return x.double().cpu().numpy()


# ---------------------------------------------------------------- writing
@pytest.mark.parametrize("n,rows,dtype,what,layout", [
    (1, 1, BF, "both", "dense"), (1, 5, F32, "both", "dense"), (2, 130, BF, "latent", "dense"),
    (33, 64, BF, "index", "dense"), (300, 384, BF, "both", "fused"), (300, 384, F32, "both", "fused"),
    (77, 256, BF, "both", "odd"), (77, 256, F32, "both", "odd"), (9, 128, F32, "index", "dense"),
    (1025, 1100, BF, "both", "dense"),
])
def test_write_is_exact(n, rows, dtype, what, layout, dev):
    g = torch.Generator().manual_seed(n)
    slots = torch.randperm(rows, generator=g)[:n].to(torch.int32)
    if n > 8:
        slots[3::5] = -1
    kv, key = activations(n, 576, 3 * n, dtype, n > 8), activations(n, 128, 3 * n + 1, dtype, n > 8)
    c = caches(rows, dev)
    before = {k: v.clone() for k, v in c.items()}
    if layout == "fused":                     # one projection's output, aligned rows
        both = torch.cat([kv, key], 1).to(dev)
        dkv, dkey = both[:, :576], both[:, 576:]
    elif layout == "odd":                     # rows that start anywhere
        dkv, dkey = wide(kv, 13, 5, dev), wide(key, 3, 1, dev)
    else:
        dkv, dkey = kv.to(dev), key.to(dev)
    args = {}
    if what != "index":
        args.update(kv=dkv, kv_q8=c["kv_q8"], kv_scale=c["kv_scale"])
    if what != "latent":
        args.update(k_idx=dkey, k_codes=c["k_codes"], k_scale=c["k_scale"])
    ws = make_ws(0, dev)
    launches = ic.kernel_launches(8)
    ic.cache_write_q8(slots.to(dev), ws, **args)
    assert ic.read_status(ws) == 0 and ic.kernel_launches(8) == launches + 1
    keep = (slots >= 0).numpy()
    at = slots.numpy()[keep]
    want = {k: v.cpu().numpy().copy() for k, v in before.items()}
    if what != "index":
        want["kv_q8"][at], want["kv_scale"][at] = u8.pack_rows(num(kv)[keep])
    if what != "latent":
        codes, scales = u8.quantise(num(key)[keep])
        want["k_codes"][at], want["k_scale"][at] = codes, scales
    for name in c:
        got = c[name].cpu().numpy()
        if name == "kv_q8":                   # NaN of the bfloat16 columns: any NaN will do
            a, b = got[:, 512:].copy().view(np.uint16), want[name][:, 512:].copy().view(np.uint16)
            nan = ((a & 0x7FFF) > 0x7F80) & ((b & 0x7FFF) > 0x7F80)
            np.testing.assert_array_equal(np.where(nan, 0, a), np.where(nan, 0, b))
            got, want[name] = got[:, :512], want[name][:, :512]
        np.testing.assert_array_equal(got, want[name], err_msg=name)


def test_write_without_slots_and_an_empty_call(dev):
    kv = activations(19, 576, 5, BF).to(dev)
    c, ws = caches(24, dev), make_ws(0, dev)
    ic.cache_write_q8(None, ws, kv=kv, kv_q8=c["kv_q8"], kv_scale=c["kv_scale"])
    rows, scales = u8.pack_rows(num(kv))
    np.testing.assert_array_equal(c["kv_q8"][:19].cpu().numpy(), rows)
    np.testing.assert_array_equal(c["kv_scale"][:19].cpu().numpy(), scales)
    assert (c["kv_q8"][19:] == 0xA5).all() and (c["kv_scale"][19:] == -3).all()
    n0 = ic.kernel_launches(0)
    ic.cache_write_q8(torch.empty(0, dtype=torch.int32, device=dev), ws, kv=kv[:0], kv_q8=c["kv_q8"],
                      kv_scale=c["kv_scale"])
    assert ic.kernel_launches(0) == n0 and ic.read_status(ws) == 0


def test_slots_outside_the_cache_are_skipped_and_flagged(dev):
    kv = activations(4, 576, 6, BF).to(dev)
    c, ws = caches(8, dev), make_ws(0, dev)
    slots = torch.tensor([2, 8, -2, 2147483647], dtype=torch.int32, device=dev)
    ic.cache_write_q8(slots, ws, kv=kv, kv_q8=c["kv_q8"], kv_scale=c["kv_scale"])
    assert ic.read_status(ws) == INDEX_RANGE
    rows, _ = u8.pack_rows(num(kv)[:1])
    np.testing.assert_array_equal(c["kv_q8"][2:3].cpu().numpy(), rows)
    untouched = [0, 1, 3, 4, 5, 6, 7]
    assert (c["kv_q8"][untouched] == 0xA5).all() and (c["kv_scale"][untouched] == -3).all()
    out = torch.full((4, 576), 5.0, dtype=BF, device=dev)
    ic.cache_read_q8(slots, ws, kv=out, kv_q8=c["kv_q8"], kv_scale=c["kv_scale"])
    assert ic.read_status(ws) == INDEX_RANGE
    assert (out[1:] == 0).all() and (out[0] != 0).any()


# ---------------------------------------------------------------- reading
@pytest.mark.parametrize("n,rows,dtype,what,layout", [
    (1, 1, BF, "both", "dense"), (3, 7, F32, "both", "dense"), (130, 256, BF, "latent", "dense"),
    (65, 128, F32, "index", "dense"), (257, 300, BF, "both", "odd"), (257, 300, F32, "both", "odd"),
    (2049, 2048, BF, "both", "dense"),
])
def test_read_is_exact(n, rows, dtype, what, layout, dev):
    g = torch.Generator().manual_seed(n)
    raw = torch.randint(0, 256, (rows, 640), generator=g, dtype=torch.uint8)
    raw[:, 512:] = activations(rows, 64, n, BF).view(torch.uint8)
    scale = 2.0 ** torch.randint(-32, 40, (rows,), generator=g).float()
    codes = torch.randint(0, 256, (rows, 128), generator=g, dtype=torch.uint8)
    key_scale = torch.rand(rows, generator=g) + 0.01           # any float32 scale
    slots = torch.randint(0, rows, (n,), generator=g, dtype=torch.int32)   # rows may repeat
    if n > 2:
        slots[1::3] = -1
    extra, offset = (13, 5) if layout == "odd" else (0, 0)
    kv = torch.full((n, 576 + extra), 7.0, dtype=dtype, device=dev)
    key = torch.full((n, 128 + extra), 7.0, dtype=dtype, device=dev)
    args = {}
    if what != "index":
        args.update(kv=kv[:, offset:offset + 576], kv_q8=raw.to(dev), kv_scale=scale.to(dev))
    if what != "latent":
        args.update(k_idx=key[:, offset:offset + 128], k_codes=codes.to(dev), k_scale=key_scale.to(dev))
    ws = make_ws(0, dev)
    ic.cache_read_q8(slots.to(dev), ws, **args)
    assert ic.read_status(ws) == 0
    at, pad = slots.clamp(min=0).long().numpy(), (slots < 0).numpy()
    want_kv = u8.unpack_rows(raw.numpy()[at], scale.numpy()[at])
    want_key = (u8.decode_e4m3(codes.numpy()[at]).astype(np.float32) * key_scale.numpy()[at][:, None])
    if dtype == BF:
        want_key = u8.bf16_value(u8.bf16_bits(want_key))
    want_kv[pad], want_key[pad] = 0.0, 0.0
    for name, got, want, used in (("kv", kv, want_kv, what != "index"),
                                  ("k_idx", key, want_key, what != "latent")):
        body = num(got[:, offset:offset + want.shape[1]])
        np.testing.assert_array_equal(body, want if used else np.full_like(want, 7.0), err_msg=name)
        rest = torch.cat([got[:, :offset], got[:, offset + want.shape[1]:]], 1)
        assert (rest == 7).all(), name


def test_rows_far_into_a_large_cache(dev):
    """Row offsets past 32 bits: a 5 GB cache, its last rows."""
    rows = 8_000_000
    c = dict(kv_q8=torch.zeros(rows, 640, dtype=torch.uint8, device=dev), kv_scale=torch.zeros(rows, device=dev))
    kv = activations(3, 576, 8, BF).to(dev)
    slots = torch.tensor([rows - 1, 6_710_887, 5], dtype=torch.int32, device=dev)
    ws = make_ws(0, dev)
    ic.cache_write_q8(slots, ws, kv=kv, **c)
    want, scales = u8.pack_rows(num(kv))
    for i, s in enumerate(slots.tolist()):
        np.testing.assert_array_equal(c["kv_q8"][s].cpu().numpy(), want[i])
    assert int((c["kv_scale"] != 0).sum()) == 3
    back = torch.empty(3, 576, dtype=F32, device=dev)
    ic.cache_read_q8(slots, ws, kv=back, **c)
    np.testing.assert_array_equal(num(back), u8.unpack_rows(want, scales))
    # attention over pages at the end of the cache
    b = Tree([4], 1, dev, seed=9, Hq=5)
    b.kv_rows(c["kv_q8"], c["kv_scale"], [rows // 128 - 1])
    out = b.run(ws=None)
    b.check(out)
    assert ic.read_status(ws) == 0


# ---------------------------------------------------------------- attention
class Tree:
    """A batch: sequences' logical quantised caches, their pages, trees and queries."""

    def __init__(self, lens, Lq, dev, seed, Hq=128, k=0, page=128, masks="tree", gain=1.0, T_max=None,
                 size=None, spare=2, holes=True):
        g = torch.Generator().manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        self.lens, self.Lq, self.Hq, self.k, self.page, self.dev = list(lens), Lq, Hq, k, page, dev
        self.B, self.T_max = len(lens), T_max or max(max(lens), Lq)
        self.scale = 576 ** -0.5
        good = [n if Lq <= n <= self.T_max else 0 for n in self.lens]
        self.good = good
        self.q = (torch.randn(self.B, Lq, Hq, 576, generator=g) * gain).to(BF)
        self.rows, self.scales, self.kv = [], [], []
        for n in good:
            x = torch.randn(max(n, 1), 576, generator=g).numpy().astype(np.float64)
            if size is not None:               # rows of very different sizes
                x *= 2.0 ** self.rng.integers(-size, size + 1, (max(n, 1), 1))
            r, s = u8.pack_rows(x)
            self.rows.append(r)
            self.scales.append(s)
        if masks is None:
            self.masks = None
        elif masks == "none":
            self.masks = np.zeros((self.B, Lq), dtype=np.uint64)
        else:
            self.masks = np.zeros((self.B, Lq), dtype=np.uint64)
            for b in range(self.B):
                for i in range(Lq):
                    up = int(self.masks[b, int(self.rng.integers(0, i))]) if i else 0
                    self.masks[b, i] = up | 1 << i
        self.idx = None
        if k:
            self.idx = np.full((self.B, Lq, k), -1, dtype=np.int32)
            for b in range(self.B):
                for i in range(Lq):
                    t = good[b] - Lq + i
                    if t < 0:
                        continue
                    pick = self.rng.permutation(t + 1)[:k]
                    at = self.rng.permutation(k)[:len(pick)] if holes else np.arange(len(pick))
                    self.idx[b, i, np.sort(at)] = np.sort(pick)
        per = [-(-n // page) for n in good]
        self.num_pages = sum(per) + spare
        order = self.rng.permutation(self.num_pages)
        self.table = np.full((self.B, -(-self.T_max // page)), -1, dtype=np.int32)
        self.cache = np.full((self.num_pages * page, 640), 0x7F, dtype=np.uint8)   # NaN where nothing lies
        self.cache[:, 512:] = 0xFF
        self.cache_scale = np.full(self.num_pages * page, np.nan, dtype=np.float32)
        c = 0
        for b in range(self.B):
            self.table[b, :per[b]] = order[c:c + per[b]]
            c += per[b]
        self.place()

    def place(self):
        for b in range(self.B):
            for s in range(self.good[b]):
                p = self.table[b, s // self.page] * self.page + s % self.page
                self.cache[p], self.cache_scale[p] = self.rows[b][s], self.scales[b][s]
        self.d_cache = torch.from_numpy(self.cache).to(self.dev)
        self.d_scale = torch.from_numpy(self.cache_scale).to(self.dev)

    def kv_rows(self, cache, scale, pages):
        """Puts the (single) sequence into given pages of a cache that is there."""
        self.num_pages, self.d_cache, self.d_scale = len(cache) // self.page, cache, scale
        self.table = np.array([pages], dtype=np.int32)
        at = torch.tensor([pages[s // self.page] * self.page + s % self.page for s in range(self.lens[0])],
                          device=self.dev)
        cache[at] = torch.from_numpy(self.rows[0]).to(self.dev)
        scale[at] = torch.from_numpy(self.scales[0]).to(self.dev)

    def device(self):
        self.d_lens = torch.tensor(self.lens, dtype=torch.int32, device=self.dev)
        self.d_table = torch.from_numpy(self.table).to(self.dev)
        self.d_tree = None if self.masks is None else torch.from_numpy(self.masks.view(np.int64)).to(self.dev)
        self.d_idx = None if self.idx is None else torch.from_numpy(self.idx).to(self.dev)
        self.pr = ic.paged_rows(self.d_lens, self.d_table, self.T_max, self.page, self.num_pages, self.Lq)
        self.d_q = self.q.to(self.dev)

    def workspace(self):
        return make_ws(ic.tree_attn_q8_workspace_size(self.pr, self.k, self.Hq), self.dev)

    def call(self, out, ws):
        ic.tree_attn_q8_paged(self.d_q, self.d_cache, self.d_scale, self.d_idx, self.pr, self.scale, out, ws,
                              tree=self.d_tree)

    def run(self, ws="new", status=0):
        self.device()
        ws = self.workspace()
        out = torch.full((self.B, self.Lq, self.Hq, 512), 3.0, dtype=BF, device=self.dev)
        n0 = ic.kernel_launches(9)
        self.call(out, ws)
        assert ic.read_status(ws) == status
        assert ic.kernel_launches(9) == n0 + 1
        return out

    def check(self, out, rows=None, hidden=()):
        """Compares rows (b, i) (default: all); `hidden`: (b, s) positions that no row can see."""
        got = num(out)
        for b in range(self.B):
            n = self.good[b]
            kv = u8.unpack_rows(self.rows[b], self.scales[b]) if n else None
            for i in range(self.Lq):
                if rows is not None and (b, i) not in rows:
                    continue
                mask = u8.chain(i) if self.masks is None else int(self.masks[b, i])
                seen = u8.seen_positions(n, self.Lq, i, mask, None if self.idx is None else self.idx[b, i])
                seen = [s for s in seen if (b, s) not in hidden]
                ref, tol = u8.attend(num(self.q[b, i]), kv, self.scales[b], seen if n else [], self.scale)
                u8.check_rows(got[b, i], ref, tol, "sequence %d, node %d" % (b, i))


@pytest.mark.parametrize("lens,Lq,Hq,page,masks", [
    ([1], 1, 1, 128, None),
    ([1, 2, 3], 1, 128, 128, "tree"),
    ([63, 64, 65, 127, 128, 129, 130, 255, 256, 257], 1, 128, 128, None),
    ([300, 37, 513], 5, 16, 128, "tree"),
    ([64, 65, 700, 191], 64, 3, 128, "tree"),
    ([200, 131], 17, 128, 256, "tree"),
    ([200, 131], 9, 67, 128, None),
    ([1000], 7, 100, 384, "tree"),
    ([5000, 129], 3, 128, 128, "tree"),
])
def test_attention_over_every_position(lens, Lq, Hq, page, masks, dev):
    b = Tree(lens, Lq, dev, seed=sum(lens) + Lq, Hq=Hq, page=page, masks=masks)
    b.check(b.run())


@pytest.mark.parametrize("lens,Lq,Hq,k,masks,holes", [
    ([1], 1, 128, 1, None, False),
    ([500, 20], 1, 128, 63, "tree", True),
    ([500, 300], 6, 128, 64, "tree", False),
    ([900, 65], 4, 16, 129, "tree", True),
    ([700], 64, 7, 100, "tree", True),
    ([3000, 2500, 40], 2, 128, 2048, "tree", False),
    ([4000], 3, 33, 2500, None, True),
    ([150], 1, 128, 5000, None, True),
])
def test_attention_over_selected_positions(lens, Lq, Hq, k, masks, holes, dev):
    b = Tree(lens, Lq, dev, seed=k, Hq=Hq, k=k, masks=masks, holes=holes)
    b.check(b.run())


def test_positions_named_twice_count_twice(dev):
    b = Tree([90], 2, dev, seed=3, Hq=9, k=40)
    b.idx[0, 0, :] = 7
    b.idx[0, 1, :20], b.idx[0, 1, 20:] = 5, 89
    b.check(b.run())


@pytest.mark.parametrize("k", [0, 200])
def test_sharp_logits(k, dev):
    b = Tree([700, 300], 3, dev, seed=21, k=k, gain=16.0)
    b.check(b.run())


@pytest.mark.parametrize("k", [0, 130])
def test_rows_of_very_different_sizes(k, dev):
    """Scales from 2^-14 to 2^6 within one sequence."""
    b = Tree([400], 4, dev, seed=22, k=k, size=10, gain=0.02, Hq=40)
    b.check(b.run())


def test_many_small_weights_beside_a_large_one(dev):
    """One position outweighs each of 6000 others by 2^16, and they hold a third of its weight together:
    none of them may be lost."""
    b = Tree([6001], 1, dev, seed=47, Hq=128)
    u = np.zeros(576)
    u[540:560] = 1.0                           # the logits come from columns that carry no value
    q = num(b.q) * 0
    q[0, 0] = u
    b.q = torch.from_numpy(q).to(BF)
    for s in range(6001):
        x = np.zeros(576)
        x[:512] = 1.0 + 0.5 * np.sin(s + np.arange(512)) if s else -1.0
        x[540:560] = 24.0 * np.log(2.0 ** 16 / 4) / 20 if s == 0 else 0.0
        r, sc = u8.pack_rows(x[None])
        b.rows[0][s], b.scales[0][s] = r[0], sc[0]
    b.place()
    b.scale = 1.0 / 24
    out = b.run()
    b.check(out)
    share = 6000 / (6000 + 2.0 ** 14)
    assert abs(float(out.float().mean()) - (2 * share - 1)) < 0.02


def test_growing_logits_rescale(dev):
    """Later positions win by ever larger steps: the running maximum moves in every block."""
    b = Tree([1500], 2, dev, seed=23, Hq=128)
    q = num(b.q)
    for s in range(1500):
        x = q[0, 0, s % 128] / np.linalg.norm(q[0, 0, s % 128]) * (s / 15.0)
        r, sc = u8.pack_rows(x[None])
        b.rows[0][s], b.scales[0][s] = r[0], sc[0]
    b.place()
    b.check(b.run())


def test_rows_that_see_nothing_are_zero(dev):
    b = Tree([6, 40], 6, dev, seed=24, Hq=20, masks="none")
    out = b.run()
    assert (out[0] == 0).all()                 # no context, no node
    b.check(out)
    b = Tree([300, 200], 3, dev, seed=25, Hq=128, k=64)
    b.idx[0, 1] = -1
    b.idx[1, 2, :], b.masks[1, 2] = 199, 1      # names a node that it does not see
    out = b.run()
    assert (out[0, 1] == 0).all() and (out[1, 2] == 0).all()
    b.check(out)


def test_what_is_out_of_range_is_skipped_and_flagged(dev):
    # a length outside [Lq, T_max]
    b = Tree([2, 50, 80, -5], 3, dev, seed=26, Hq=10, T_max=64)
    out = b.run(status=INDEX_RANGE)
    assert (out[0] == 0).all() and (out[2] == 0).all() and (out[3] == 0).all()
    b.check(out)
    # an index outside the sequence
    b = Tree([70, 300], 2, dev, seed=27, Hq=128, k=66)
    b.idx[0, 0, :3] = [70, -2, 2147483647]
    b.check(b.run(status=INDEX_RANGE))
    # a page outside the cache hides its positions
    for k, page_no in ((0, 99), (150, -7)):
        b = Tree([400, 200], 2, dev, seed=28, Hq=17, k=k)
        if k:
            b.idx[0] = np.arange(100, 250)
        b.table[0, 1] = page_no
        b.check(b.run(status=INDEX_RANGE), hidden={(0, s) for s in range(128, 256)})


@pytest.mark.parametrize("k,Hq", [(0, 10), (0, 128), (100, 10)])
def test_nan_stays_where_it_is_seen(k, Hq, dev):
    """NaN codes and infinities in a node's cache row reach the rows that see it, and no other."""
    b = Tree([200], 5, dev, seed=29, Hq=Hq, k=k)
    b.masks[0] = [1, 3, 1 | 4, 1 | 8, 1 | 2 | 16]
    if k:
        for i in range(5):
            b.idx[0, i, :60], b.idx[0, i, 60:65], b.idx[0, i, 65:] = np.arange(60), np.arange(195, 200), -1
    b.rows[0][196, 5] = 0x7F                   # node 1: a NaN code among the values
    b.rows[0][198, 600:602] = [0x80, 0x7F]     # node 3: an infinity among the last columns
    b.place()
    out = b.run()
    assert torch.isnan(out[0, 1]).all() and torch.isnan(out[0, 4]).all()
    got = num(out)
    assert np.isfinite(got[0, [0, 2]]).all()
    b.check(out, rows={(0, 0), (0, 2)})


def test_a_nan_query_stays_in_its_head(dev):
    b = Tree([150], 2, dev, seed=30, Hq=6)
    b.q[0, 1, 2, 100] = float("nan")
    b.q[0, 0, 4, 570] = float("inf")
    out = b.run()
    assert torch.isnan(out[0, 1, 2]).all() and torch.isnan(out[0, 0, 4]).all()
    assert int(torch.isnan(out).any(-1).sum()) == 2


def test_zero_query_gives_the_mean(dev):
    b = Tree([333], 2, dev, seed=31, Hq=128, masks=None)
    b.q.zero_()
    out = num(b.run())
    kv = u8.unpack_rows(b.rows[0], b.scales[0])
    for i in range(2):
        mean = kv[:332 + i, :512].mean(0)
        tol = 2.0 ** -8 * np.abs(mean) + 2.0 ** -8 * np.abs(kv[:332 + i, :512]).mean(0)
        assert (np.abs(out[0, i] - mean) <= tol).all()


@pytest.mark.parametrize("k", [0, 300])
def test_results_do_not_depend_on_the_run(k, dev):
    """The same call twice, on another stream, and replayed from a graph: the same bits."""
    b = Tree([2000, 700, 90], 4, dev, seed=32, k=k)
    first = b.run()
    ws = b.workspace()
    out = torch.empty_like(first)
    b.call(out, ws)
    assert torch.equal(out, first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2, ws2 = torch.empty_like(first), b.workspace()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        b.call(out2, ws2)
        graph = torch.cuda.CUDAGraph()
        out3 = torch.zeros_like(first)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            b.call(out3, ws2)
            b.call(out2, ws2)                  # the same workspace, one after the other
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out2, first) and torch.equal(out3, first)
    assert ic.read_status(ws) == 0 and ic.read_status(ws2) == 0


@pytest.mark.parametrize("lens,Lq,k", [([6000, 2300, 700], 8, 0), ([4000] * 6, 4, 2048)])
def test_growing_maxima_give_the_same_bits_every_time(lens, Lq, k, dev):
    """A few positions far above the others raise the running maxima again and again, in every phase of the
    blocks that are under way: each of 150 calls must give what the first gave."""
    b = Tree(lens, Lq, dev, seed=48, k=k)
    for rows, scales in zip(b.rows, b.scales):
        for s in b.rng.permutation(len(rows))[:len(rows) // 40]:
            scales[s] *= 2.0 ** int(b.rng.integers(1, 5))
    b.place()
    first = b.run()
    b.check(first, rows={(0, 0), (0, Lq - 1), (2, 1)})
    ws, out = b.workspace(), torch.empty_like(first)
    for _ in range(150):
        b.call(out, ws)
        assert torch.equal(out, first)
    assert ic.read_status(ws) == 0


def test_two_calls_at_once_on_two_streams(dev):
    a, b = Tree([3000, 800], 2, dev, seed=33, k=500), Tree([2500], 8, dev, seed=34, Hq=64)
    wa, wb = a.run(), b.run()
    oa, ob = torch.empty_like(wa), torch.empty_like(wb)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    wsa, wsb = a.workspace(), b.workspace()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(sa):
            a.call(oa, wsa)
        with torch.cuda.stream(sb):
            b.call(ob, wsb)
    torch.cuda.synchronize()
    assert torch.equal(oa, wa) and torch.equal(ob, wb)


def test_a_full_gpu_of_rows(dev):
    """More rows than the GPU holds at once: every one of them is right."""
    b = Tree([150] * 40, 6, dev, seed=35, Hq=128, k=70)
    out = b.run()
    b.check(out, rows={(0, 0), (7, 5), (20, 3), (39, 5)})
    again = b.run()
    assert torch.equal(out, again)
    one = Tree([150] * 40, 6, dev, seed=35, Hq=128, k=70)
    for name in ("lens", "good", "rows", "scales"):
        setattr(one, name, getattr(one, name)[39:])
    one.B, one.q, one.idx, one.masks, one.table = 1, one.q[39:], one.idx[39:], one.masks[39:], one.table[39:]
    alone = one.run()
    np.testing.assert_allclose(num(alone[0]), num(out[39]), rtol=2.0 ** -6, atol=2.0 ** -8)


def test_more_lists_than_the_gpu_has_pairs(dev):
    """80 lists of 16 blocks: the CTA pairs take equal runs over the lists' borders; most blocks name nothing."""
    b = Tree([40 + 3 * i for i in range(80)], 1, dev, seed=42, Hq=33, k=2048)
    b.check(b.run(), rows={(i, 0) for i in (0, 1, 2, 17, 36, 37, 38, 55, 78, 79)})


def test_a_list_over_many_pairs(dev):
    b = Tree([20000], 1, dev, seed=43, Hq=5, k=16384)
    b.check(b.run())


@pytest.mark.parametrize("lens,Lq,Hq,T_max", [
    ([64 + 61 * i for i in range(40)], 16, 16, None),       # 80 units over all pairs, several in one
    ([9000, 20, 17, 4000], 8, 16, 100000),                  # shares by length; a bound far above the lengths
    ([17] * 33 + [6000] * 3, 1, 128, 6001),                 # more sequences than lanes of a warp
    ([3] * 100, 3, 128, None),                              # units of one block
])
def test_sharing_out_by_length(lens, Lq, Hq, T_max, dev):
    b = Tree(lens, Lq, dev, seed=44, Hq=Hq, T_max=T_max)
    rows = {(i, j) for i in (0, 1, len(lens) // 2, len(lens) - 2, len(lens) - 1) for j in (0, Lq - 1)}
    b.check(b.run(), rows=rows)


@pytest.mark.parametrize("k", [0, 256])
def test_a_captured_call_follows_its_inputs(k, dev):
    """The same graph replayed after the lengths, pages, trees and queries have changed in place."""
    first = Tree([900, 40, 300], 4, dev, seed=45, Hq=48, k=k, T_max=2500)
    then = Tree([30, 2500, 4], 4, dev, seed=46, Hq=48, k=k, T_max=2500)
    want = [first.run().clone(), then.run().clone()]
    rows = max(len(first.d_cache), len(then.d_cache))
    cache = torch.zeros(rows, 640, dtype=torch.uint8, device=dev)
    scale = torch.ones(rows, device=dev)
    lens, table = first.d_lens.clone(), first.d_table.clone()
    q, tree, idx = first.d_q.clone(), first.d_tree.clone(), None if not k else first.d_idx.clone()
    pr = ic.paged_rows(lens, table, 2500, 128, rows // 128, 4)
    ws = make_ws(ic.tree_attn_q8_workspace_size(pr, k, 48), dev)
    out = torch.zeros_like(want[0])

    def call():
        ic.tree_attn_q8_paged(q, cache, scale, idx, pr, first.scale, out, ws, tree=tree)

    cache[:len(first.d_cache)], scale[:len(first.d_cache)] = first.d_cache, first.d_scale
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.synchronize()
    for turn in (1, 0, 1):
        b = (first, then)[turn]
        cache[:len(b.d_cache)], scale[:len(b.d_cache)] = b.d_cache, b.d_scale
        for mine, theirs in ((lens, b.d_lens), (table, b.d_table), (q, b.d_q), (tree, b.d_tree)) + (((idx, b.d_idx),) if k else ()):
            mine.copy_(theirs)
        out.fill_(9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[turn])
    assert ic.read_status(ws) == 0


# ---------------------------------------------------------------- refusals
def test_calls_refuse_wrong_tensors(dev):
    """Real tensors take the short way through the binding; what is wrong with one is said all the same."""
    kv, c, ws = torch.zeros(4, 576, dtype=BF, device=dev), caches(8, dev), make_ws(0, dev)
    slots = torch.arange(4, dtype=torch.int32, device=dev)
    good = dict(kv=kv, kv_q8=c["kv_q8"], kv_scale=c["kv_scale"])
    n0 = ic.kernel_launches(0)
    for bad, match in ((dict(kv=kv.half()), "kv: unexpected dtype"), (dict(kv=kv.cpu()), "kv: expected a tensor on"),
                       (dict(kv=kv.t().contiguous().t()), "kv: expected a contiguous"),
                       (dict(kv=kv[:1].expand(4, 576)), "kv: expected a contiguous"),
                       (dict(kv_q8=c["kv_q8"][:, :512]), "kv_q8: expected shape"),
                       (dict(kv_q8=torch.zeros(8, 1280, dtype=torch.uint8, device=dev)[:, :640]), "kv_q8: expected a contiguous"),
                       (dict(kv_scale=c["kv_scale"].double()), "kv_scale: unexpected dtype"),
                       (dict(kv_scale=None), "go together"), (dict(k_codes=c["k_codes"]), "go together")):
        for call in (ic.cache_write_q8, ic.cache_read_q8):
            with pytest.raises(ValueError, match=match):
                call(slots, ws, **{**good, **bad})
    with pytest.raises(ValueError, match="slots: unexpected dtype"):
        ic.cache_write_q8(slots.long(), ws, **good)
    with pytest.raises(ic.IcError):
        ic.cache_write_q8(None, ws, kv=torch.zeros(9, 576, dtype=BF, device=dev), kv_q8=c["kv_q8"], kv_scale=c["kv_scale"])
    with pytest.raises(ic.IcError):
        ic.cache_write_q8(slots, ws[:128], **good)
    b = Tree([50], 2, dev, seed=41, Hq=4)
    b.device()
    out, aws = torch.empty(1, 2, 4, 512, dtype=BF, device=dev), b.workspace()
    for name, x, match in (("d_q", b.d_q.float(), "q: unexpected dtype"), ("d_cache", b.d_cache[1:], "kv_q8: expected shape"),
                           ("d_scale", b.d_scale[::2].repeat(2)[1:], "kv_scale: expected shape"),
                           ("d_tree", b.d_tree.int(), "tree: unexpected dtype"),
                           ("d_q", b.d_q.transpose(1, 2).contiguous().transpose(1, 2), "q: expected a contiguous")):
        keep = getattr(b, name)
        setattr(b, name, x)
        with pytest.raises(ValueError, match=match):
            b.call(out, aws)
        setattr(b, name, keep)
    with pytest.raises(ic.IcError):
        b.call(out, aws[:512])
    assert ic.kernel_launches(0) == n0 and ic.read_status(ws) == 0


# ---------------------------------------------------------------- together
def test_a_serving_step_from_write_to_attention(dev):
    """A prompt and then a tree of drafted tokens are written into the pages,
    the FP8 indexer selects each node's positions from the written keys, the
    attention reads them; the cache read back gives the same through the
    bfloat16 attention."""
    g = torch.Generator().manual_seed(40)
    P, Lq, k, lens = 128, 4, 256, [700, 391]
    B, T_max = 2, 700
    pages = [6, 4]
    order = torch.randperm(12, generator=g)
    table = torch.full((B, 6), -1, dtype=torch.int32)
    table[0], table[1, :4] = order[:6].to(torch.int32), order[6:10].to(torch.int32)
    rows = 12 * P
    c = dict(kv_q8=torch.zeros(rows, 640, dtype=torch.uint8, device=dev), kv_scale=torch.zeros(rows, device=dev),
             k_codes=torch.zeros(rows, 128, dtype=torch.uint8, device=dev), k_scale=torch.zeros(rows, device=dev))
    x = torch.randn(sum(lens), 704, generator=g).to(BF).to(dev)
    d_table, d_lens = table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    where, seq = [], []
    for b in range(B):
        s = torch.arange(lens[b])
        where.append((table[b].long()[s // P] * P + s % P).to(torch.int32))
        seq += [b] * lens[b]
    slots = torch.cat(where).to(dev)
    ws = make_ws(0, dev)
    start = [0, lens[0]]
    prompt = torch.cat([torch.arange(start[b], start[b] + lens[b] - Lq) for b in range(B)]).to(dev)
    nodes = torch.cat([torch.arange(start[b] + lens[b] - Lq, start[b] + lens[b]) for b in range(B)]).to(dev)
    for part in (prompt, nodes):               # the prompt first, then the step's drafted tokens
        part_x = x[part]
        ic.cache_write_q8(slots[part], ws, kv=part_x[:, :576], k_idx=part_x[:, 576:], **c)
    # selection: each row's candidates are 0..t; the nodes that a row does not see get the lowest score
    pr = ic.paged_rows(d_lens, d_table, T_max, P, 12, Lq)
    H = 64
    from cross_layer_top_full_b200 import synth
    qi, q_scale = synth.fp8_per_token((torch.randn(B, Lq, H, 128, generator=g) / 11.3).to(dev), 2)
    w = (torch.randn(B, Lq, H, generator=g) / 8).to(dev)
    scores = torch.zeros(B, Lq, 700, device=dev)
    ic.indexer_scores_paged(qi, w, c["k_codes"], pr, scores, ws, q_scale=q_scale, k_scale_pages=c["k_scale"],
                            dtype=ic.FP8_E4M3)
    masks = np.array([[1, 3, 5, 11], [1, 3, 7, 9]], dtype=np.int64)
    for b in range(B):
        for i in range(Lq):
            for a in range(i + 1):
                if not masks[b, i] >> a & 1:
                    scores[b, i, lens[b] - Lq + a] = float("-inf")
    idx = torch.full((B, Lq, k), -1, dtype=torch.int32, device=dev)
    ic.topk_varlen(scores, pr, k, idx, ws)
    q = torch.randn(B, Lq, 128, 576, generator=g).to(BF).to(dev)
    out = torch.empty(B, Lq, 128, 512, dtype=BF, device=dev)
    aws = make_ws(ic.tree_attn_q8_workspace_size(pr, k, 128), dev)
    ic.tree_attn_q8_paged(q, c["kv_q8"], c["kv_scale"], idx, pr, 576 ** -0.5, out, aws,
                          tree=torch.from_numpy(masks).to(dev))
    assert ic.read_status(ws) == 0 and ic.read_status(aws) == 0
    hx, hs, hidx = num(x), host64(scores), idx.cpu().numpy()
    for b in range(B):
        mine = hx[start[b]:start[b] + lens[b]]
        packed, sc = u8.pack_rows(mine[:, :576])
        at = where[b].long().to(dev)
        np.testing.assert_array_equal(c["kv_q8"][at].cpu().numpy(), packed)
        codes, ks = u8.quantise(mine[:, 576:])
        np.testing.assert_array_equal(c["k_codes"][at].cpu().numpy(), codes)
        key = u8.decode_e4m3(codes) * ks[:, None]
        query = u8.decode_e4m3(qi[b].cpu().numpy()) * num(q_scale[b])[:, None, None]
        for i in range(Lq):
            t = lens[b] - Lq + i
            ref = np.maximum(query[i] @ key[:t + 1].T, 0.0)
            ref = num(w[b, i]) @ ref
            live = np.isfinite(hs[b, i, :t + 1])
            np.testing.assert_allclose(hs[b, i, :t + 1][live], ref[live], rtol=0, atol=1e-4 * np.abs(ref).max() + 1e-5)
            seen = u8.seen_positions(lens[b], Lq, i, int(masks[b, i]), hidx[b, i])
            assert len(seen) == k              # nothing was selected that the row cannot see
            a_ref, tol = u8.attend(num(q[b, i]), u8.unpack_rows(packed, sc), sc, seen, 576 ** -0.5)
            u8.check_rows(num(out[b, i]), a_ref, tol, "sequence %d, node %d" % (b, i))
    # the cache read back, through the bfloat16 attention (a tree that is a chain there: the lists name only seen nodes)
    dense = torch.zeros(B, 700, 576, dtype=BF, device=dev)
    for b in range(B):
        ic.cache_read_q8(where[b].to(dev), ws, kv=dense[b, :lens[b]], kv_q8=c["kv_q8"], kv_scale=c["kv_scale"])
        r = (1, Lq, lens[b] - Lq, 700)
        bws = make_ws(ic.sparse_attn_workspace_size(r, k, 128, 576, 512, ic.BF16), dev)
        ref = torch.empty(1, Lq, 128, 512, dtype=BF, device=dev)
        ic.sparse_attn(q[b:b + 1], dense[b], 576, dense[b], 576, idx[b:b + 1], r, 512, 576 ** -0.5, ref, bws)
        assert ic.read_status(bws) == 0
        check_attention(num(out[b:b + 1]), num(ref), "read back, sequence %d" % b)
    assert ic.read_status(ws) == 0
