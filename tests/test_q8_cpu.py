"""The quantised cache without a GPU: pins of the 64-bit numpy definition that
the GPU tests compare with, and every refusal of the C ABI and the binding."""
import ctypes

import numpy as np
import pytest
import torch

import cross_layer_top_full_b200 as ic
import q8_util as u8


# ---------------------------------------------------------------- the definition
def test_e4m3_decode_matches_torch_for_every_code():
    c = torch.arange(256, dtype=torch.uint8)
    want = c.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(u8.decode_e4m3(c.numpy()), want)


def test_e4m3_encode_matches_torch_in_range_and_saturates():
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(4000, generator=g) * 100, torch.randn(4000, generator=g) / 64,
                   torch.tensor([0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9, 17.0, 19.0, 448.0])])
    x = x.clamp(-448, 448)
    np.testing.assert_array_equal(u8.encode_e4m3(x.numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    got = u8.encode_e4m3([1e9, -1e9, np.inf, -np.inf, np.nan, 460.0])
    assert list(got) == [126, 254, 126, 254, 127, 126]


def test_scale_borders():
    def s(top):
        x = np.zeros(512)
        x[7] = top
        return u8.row_scale(x[None])[0]
    assert s(0.0) == 1.0 and s(448.0) == 1.0 and s(np.nextafter(448.0, 500)) == 2.0
    assert s(224.0) == 0.5 and s(225.0) == 1.0 and s(-1.75) == 2.0 ** -8
    assert s(1e-30) == 2.0 ** -32 and s(448.0 * 2.0 ** -32) == 2.0 ** -32
    assert s(np.inf) == 1.0 and s(np.nan) == 1.0 and s(3e38) == 2.0 ** 120


def test_pack_and_unpack_round_trip():
    rng = np.random.default_rng(0)
    kv = rng.standard_normal((20, 576)) * np.exp(rng.standard_normal((20, 1)))
    rows, scales = u8.pack_rows(kv)
    back = u8.unpack_rows(rows, scales)
    # 4 significant bits (half a step 2^-4 relative), a floor of half the smallest step
    err = np.abs(back[:, :512] - kv[:, :512])
    assert (err <= np.maximum(2.0 ** -4 * np.abs(kv[:, :512]), 2.0 ** -10 * scales[:, None])).all()
    assert (np.abs(back[:, 512:] - kv[:, 512:]) <= 2.0 ** -8 * np.abs(kv[:, 512:])).all()
    rows2, scales2 = u8.pack_rows(back)
    np.testing.assert_array_equal(rows2, rows)


def test_tree_reading():
    # 6 positions, the last 3 are nodes: node 2 sees node 0 and itself
    assert u8.seen_positions(6, 3, 2, 0b101, None) == [0, 1, 2, 3, 5]
    assert u8.seen_positions(6, 3, 2, 0b101, [5, 4, -1, 1, 1, 9]) == [5, 1, 1]
    assert u8.seen_positions(3, 3, 0, 0, None) == []
    assert [u8.chain(i) for i in (0, 2)] == [1, 7]


# ---------------------------------------------------------------- C ABI refusals
class _Host:
    """Aligned host memory standing in for a device buffer that no launch will touch."""

    def __init__(self, nbytes):
        self.raw = (ctypes.c_char * (nbytes + 256))()
        self.addr = (ctypes.addressof(self.raw) + 255) // 256 * 256


@pytest.fixture(scope="module")
def lib():
    return ic.lib()


@pytest.mark.parametrize("which", ["write", "read"])
def test_cache_calls_refuse_bad_arguments(lib, which):
    ws = _Host(512)
    P = 4096                                   # an aligned address that nothing reads

    def call(kv=P, kvs=576, ki=P, kis=128, dt=ic.BF16, n=4, slots=P, q=P, s=P, c=P, cs=P, rows=8,
             w=ws.addr, wb=512):
        if which == "write":
            return lib.ic_cache_write_q8(kv, kvs, ki, kis, dt, n, slots, q, s, c, cs, rows, w, wb, None)
        return lib.ic_cache_read_q8(q, s, c, cs, rows, n, slots, dt, kv, kvs, ki, kis, w, wb, None)

    before = ic.kernel_launches(0)
    assert call(dt=ic.FP8_E4M3) == -1 and call(dt=7) == -1
    assert call(n=-1) == -1 and call(rows=-1) == -1 and call(n=1 << 31) == -1 and call(rows=1 << 31) == -1
    assert call(kvs=575) == -1 and call(kis=127) == -1
    assert call(kv=None, ki=None) == -1
    assert call(q=None) == -1 and call(s=None) == -1 and call(c=None) == -1 and call(cs=None) == -1
    assert call(kv=None) == -1 and call(ki=None) == -1          # the others of the pair are there
    assert call(q=P + 8) == -1 and call(c=P + 8) == -1          # 16-byte alignment
    assert call(s=P + 2) == -1 and call(cs=P + 2) == -1
    assert call(kv=P + 1) == -1 and call(ki=P + 1) == -1 and call(kv=P + 2, dt=ic.F32) == -1
    assert call(slots=None, n=9) == -1                          # more rows than the cache has
    assert call(w=None) == -4 and call(wb=255) == -4 and call(w=ws.addr + 16) == -4
    # nothing to do: no pointer is looked at
    assert call(n=0, kv=None, ki=None, q=None, s=None, c=None, cs=None, slots=None, rows=0) == 0
    assert ic.kernel_launches(0) == before


def test_tree_attention_refuses_bad_arguments(lib):
    ws = _Host(4096)
    P = 4096

    def pr(**kw):
        d = dict(B=2, Lq=2, T_max=512, seq_lens=P, block_table=P, max_pages=4, page_size=128, num_pages=8)
        d.update(kw)
        return ic.PagedRows(*[d[n] for n, _ in ic.PagedRows._fields_])

    def call(p=None, q=P, kv=P, s=P, idx=P, k=64, tree=P, Hq=8, out=P, w=ws.addr, wb=None):
        p = p or pr()
        if wb is None:
            wb = 1 << 40                       # a size only; nothing is touched
        return lib.ic_tree_attn_q8_paged(q, kv, s, idx, k, tree, ctypes.byref(p), Hq, 0.1, out, w, wb, None)

    before = ic.kernel_launches(0)
    assert call(pr(Lq=65)) == -1 and call(pr(Lq=0)) == -1       # nodes
    assert call(pr(page_size=64)) == -1 and call(pr(max_pages=3)) == -1 and call(pr(num_pages=0)) == -1
    assert call(pr(T_max=1)) == -1 and call(pr(seq_lens=None)) == -1 and call(pr(block_table=None)) == -1
    assert call(Hq=0) == -1 and call(Hq=129) == -1
    assert call(k=-1) == -1 and call(k=16385) == -1
    assert call(k=0) == -1 and call(idx=None) == -1             # idx and k go together
    assert call(q=None) == -1 and call(kv=None) == -1 and call(s=None) == -1 and call(out=None) == -1
    assert call(q=P + 2) == -1 and call(kv=P + 8) == -1 and call(out=P + 4) == -1
    assert call(tree=P + 4) == -1 and call(idx=P + 2) == -1 and call(s=P + 1) == -1
    assert call(w=None) == -4 and call(wb=16) == -4 and call(w=ws.addr + 64) == -4
    assert lib.ic_tree_attn_q8_paged(P, P, P, P, 64, P, None, 8, 0.1, P, ws.addr, 4096, None) == -1
    empty = pr(B=0, seq_lens=None, block_table=None)
    assert call(empty, q=None, kv=None, s=None, idx=None, k=0, tree=None, out=None) == 0
    assert ic.kernel_launches(0) == before
    assert ic.tree_attn_q8_workspace_size(pr(), 64, 8) >= ic.STATUS_BYTES
    for bad in (pr(Lq=65), pr(B=0), pr(T_max=0)):
        assert ic.tree_attn_q8_workspace_size(bad, 64, 8) == ic.STATUS_BYTES
    assert ic.tree_attn_q8_workspace_size(pr(), -1, 8) == ic.STATUS_BYTES
    assert int(lib.ic_tree_attn_q8_workspace_size(None, 64, 8)) == ic.STATUS_BYTES


# ---------------------------------------------------------------- binding refusals
class _Dev:
    """What the binding asks of a CUDA tensor."""

    def __init__(self, *shape, dtype=torch.uint8, index=0, strides=None, cuda=True):
        self.shape, self.dtype, self.is_cuda = shape, dtype, cuda
        self.device = torch.device("cuda", index) if cuda else torch.device("cpu")
        n, dense = 1, []
        for s in reversed(shape):
            dense.insert(0, n)
            n *= s
        self.strides = tuple(strides or dense)
        self.dense = self.strides == tuple(dense)

    def get_device(self):
        return self.device.index if self.is_cuda else -1

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self.strides

    def is_contiguous(self):
        return self.dense

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def device0(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


@pytest.mark.parametrize("call", [ic.cache_write_q8, ic.cache_read_q8])
def test_binding_checks_cache_tensors(lib, device0, call):
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    good = dict(kv=_Dev(4, 576, dtype=bf), kv_q8=_Dev(8, 640), kv_scale=_Dev(8, dtype=f32),
                k_idx=_Dev(4, 128, dtype=bf), k_codes=_Dev(8, 128), k_scale=_Dev(8, dtype=f32))
    slots, ws = _Dev(4, dtype=i32), _Dev(256)
    before = ic.kernel_launches(0)

    def refused(match, slots=slots, ws=ws, **kw):
        with pytest.raises(ValueError, match=match):
            call(slots, ws, **{**good, **kw})

    refused("kv: expected a tensor on cuda:0", kv=_Dev(4, 576, dtype=bf, cuda=False))
    refused("kv_q8: expected a tensor on cuda:0", kv_q8=_Dev(8, 640, index=1))
    refused("kv: unexpected dtype", kv=_Dev(4, 576, dtype=torch.float16))
    refused("k_idx: unexpected dtype", k_idx=_Dev(4, 128, dtype=f32))       # not kv's type
    refused("kv: expected shape", kv=_Dev(4, 512, dtype=bf))
    refused("kv: expected a contiguous tensor .* or rows", kv=_Dev(4, 576, dtype=bf, strides=(1, 4)))
    refused("kv: expected a contiguous tensor .* or rows", kv=_Dev(1, 576, dtype=bf, strides=(576, 2)), k_idx=None,
            k_codes=None, k_scale=None)
    refused("kv: expected a contiguous tensor .* or rows", kv=_Dev(4, 576, dtype=bf, strides=(0, 1)))  # one row for all
    refused("k_idx: expected shape", k_idx=_Dev(5, 128, dtype=bf))
    refused("kv_q8: expected shape", kv_q8=_Dev(8, 656))
    refused("kv_q8: expected a contiguous", kv_q8=_Dev(8, 640, strides=(1280, 1)))
    refused("kv_scale: expected shape", kv_scale=_Dev(7, dtype=f32))
    refused("k_codes: expected shape", k_codes=_Dev(9, 128))
    refused("slots: expected shape", slots=_Dev(5, dtype=i32))
    refused("slots: unexpected dtype", slots=_Dev(4, dtype=torch.int64))
    refused("ws: unexpected dtype", ws=_Dev(256, dtype=f32))
    refused("kv, kv_q8 and kv_scale go together", kv=None)
    refused("kv, kv_q8 and kv_scale go together", kv_scale=None)
    refused("k_idx, k_codes and k_scale go together", k_codes=None)
    refused("k_idx, k_codes and k_scale go together", k_idx=None)
    with pytest.raises(ValueError, match="give kv, k_idx or both"):
        call(slots, ws)
    assert ic.kernel_launches(0) == before


def test_binding_checks_tree_attention_tensors(lib, device0):
    bf, f32, i32, i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
    pr = ic.PagedRows(2, 3, 256, 4096, 4096, 2, 128, 4)
    good = dict(q=_Dev(2, 3, 16, 576, dtype=bf), kv_q8=_Dev(512, 640), kv_scale=_Dev(512, dtype=f32),
                idx=_Dev(2, 3, 64, dtype=i32), out=_Dev(2, 3, 16, 512, dtype=bf), ws=_Dev(1 << 30),
                tree=_Dev(2, 3, dtype=i64))
    before = ic.kernel_launches(0)

    def refused(match, **kw):
        a = {**good, **kw}
        with pytest.raises(ValueError, match=match):
            ic.tree_attn_q8_paged(a["q"], a["kv_q8"], a["kv_scale"], a["idx"], pr, 0.1, a["out"], a["ws"],
                                  tree=a["tree"])

    refused("q: expected shape", q=_Dev(2, 2, 16, 576, dtype=bf))
    refused("q: unexpected dtype", q=_Dev(2, 3, 16, 576, dtype=f32))
    refused("q: expected shape", q=_Dev(6, 16, 576, dtype=bf))
    refused("q: expected a contiguous", q=_Dev(2, 3, 16, 576, dtype=bf, strides=(3 * 16 * 600, 16 * 600, 600, 1)))
    refused("q: expected a tensor on cuda:0", q=_Dev(2, 3, 16, 576, dtype=bf, index=1))
    refused("kv_q8: expected shape", kv_q8=_Dev(511, 640))
    refused("kv_scale: expected shape", kv_scale=_Dev(511, dtype=f32))
    refused("idx: expected shape", idx=_Dev(2, 1, 64, dtype=i32))
    refused("idx: unexpected dtype", idx=_Dev(2, 3, 64, dtype=i64))
    refused("idx: names no position", idx=_Dev(2, 3, 0, dtype=i32))
    refused("tree: unexpected dtype", tree=_Dev(2, 3, dtype=i32))
    refused("tree: expected shape", tree=_Dev(2, 4, dtype=i64))
    refused("out: expected shape", out=_Dev(2, 3, 15, 512, dtype=bf))
    refused("ws: expected a tensor on cuda:0", ws=_Dev(1 << 20, cuda=False))
    assert ic.kernel_launches(0) == before


def test_the_short_way_declines_what_is_not_plainly_right(lib):
    """csrc/fastcall.cpp makes a call only of plain CUDA tensors; anything else goes the long way."""
    fast = ic._torch_names().fast
    assert fast is not None, "build _fastcall.so: python -m cross_layer_top_full_b200.build"
    before = ic.kernel_launches(0)
    cpu, dev = torch.zeros(4, 576, dtype=torch.bfloat16), _Dev(4, 576, dtype=torch.bfloat16)
    for kv in (None, cpu, dev, "kv", cpu.numpy):
        for call in (fast.cache_write_q8, fast.cache_read_q8):
            assert call(None, torch.zeros(256, dtype=torch.uint8), kv, kv, kv, None, None, None, 0, 0) is None
    assert fast.cache_write_q8(None, None) is None                # a wrong number of arguments
    pr = ic.PagedRows(1, 1, 8, 4096, 4096, 1, 128, 1)
    for x in (None, cpu, dev):
        assert fast.tree_attn_q8(x, x, x, None, None, pr, 0.1, x, x, 0, 0) is None
        assert fast.tree_attn_q8(x, x, x, None, None, b"short", 0.1, x, x, 0, 0) is None
        assert fast.tree_attn_q8(x, x, x, None, None, pr, "scale", x, x, 0, 0) is None
    with pytest.raises(TypeError):
        fast.bind(1)
    assert ic.kernel_launches(0) == before
