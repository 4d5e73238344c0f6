"""Cases of the quantised latent cache: writing it, reading it back, and the
attention of drafted tokens over it.

A token's latent row of 576 values is kept as 640 bytes and one float32 scale s
in an array of its own: 512 e4m3 codes and 64 bfloat16 values, all of them
divided by s.  Its indexer key is kept as 128 e4m3 codes and one float32 scale
likewise.  A scale is the smallest power of two s >= 2^-32 with absmax <= 448 s
over the coded columns' finite values (1 where they are all 0): dividing by it
and multiplying with it are exact.

  write   rows [n, 576] and indexer keys [n, 128] go to the physical rows
          slots[n] of the caches (-1: skipped)
  read    the reverse: rows slots[n] of the caches as bfloat16 or float32
          (-1: zeros)
  attend  each sequence's last `nodes` cached tokens are a tree of drafted
          tokens; a node's query sees the positions before the tree (all of
          them, or those that its index list names) and the nodes of its
          bit mask
"""
import math
import random

import torch

own = False

ROW, WIDTH, VALUES, KEYS = 640, 576, 512, 128
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the step of a decode batch of 32 sequences: one token each, latent and indexer key
        {"name": "write_decode_32", "op": "write", "n": 32, "rows": 65536, "dtype": "bf16", "what": "both", "pad": 0},
        # a prompt of 8192 tokens, the fused projection's output, in pages out of order
        {"name": "write_prompt_8k", "op": "write", "n": 8192, "rows": 16384, "dtype": "bf16", "what": "both", "pad": 0},
        # a layer without an indexer, float32 activations, a padded batch
        {"name": "write_shared_f32", "op": "write", "n": 3001, "rows": 8192, "dtype": "f32", "what": "latent", "pad": 9},
        # the whole context of a long sequence, moved into the cache at once
        {"name": "write_context_64k", "op": "write", "n": 65536, "rows": 65536, "dtype": "bf16", "what": "both", "pad": 0},
        # a short shared prefix read back in front of a chunk of a prompt
        {"name": "read_prefix_509", "op": "read", "n": 509, "rows": 16384, "dtype": "bf16", "what": "both", "pad": 0},
        # a padded batch read back for a float32 layer
        {"name": "read_padded_f32", "op": "read", "n": 4999, "rows": 16384, "dtype": "f32", "what": "latent", "pad": 7},
        # the cached context of a long sequence, read back for its next chunk
        {"name": "read_context_64k", "op": "read", "n": 65536, "rows": 131072, "dtype": "bf16", "what": "latent", "pad": 0},
        # one sequence, one new token, the selected keys only: latency
        {"name": "attend_one", "op": "attend", "B": 1, "nodes": 1, "T": 32768, "k": 2048, "heads": 128, "page": 128, "tree": False},
        # the decode batch: 32 sequences of different lengths, one new token each
        {"name": "attend_batch_32", "op": "attend", "B": 32, "nodes": 1, "T": 32768, "k": 2048, "heads": 128, "page": 128, "tree": False},
        # 8 long sequences, each with a tree of 16 drafted tokens, selected keys
        {"name": "attend_tree_200k", "op": "attend", "B": 8, "nodes": 16, "T": 200000, "k": 2048, "heads": 128, "page": 256, "tree": True},
        # sequences shorter than the selection: every position counts
        {"name": "attend_dense_8k", "op": "attend", "B": 8, "nodes": 16, "T": 8192, "k": 0, "heads": 128, "page": 128, "tree": True},
        # the heads of one of eight ranks, an odd number of drafted tokens, short contexts
        {"name": "attend_dense_16_heads", "op": "attend", "B": 5, "nodes": 23, "T": 2047, "k": 0, "heads": 16, "page": 128, "tree": True},
    ]


def spread(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend"])
    if op != "attend":
        n = spread(rng, 1, 65536)
        return {"op": op, "n": n, "rows": 128 * rng.randint(-(-n // 128), -(-n // 128) + 512),
                "dtype": rng.choice(["bf16", "bf16", "f32"]) if n <= 30000 else "bf16",
                "what": rng.choice(["both", "latent", "index"]), "pad": rng.choice([0, 0, 3, 16])}
    while True:
        page = rng.choice([128, 256])
        c = {"op": op, "B": spread(rng, 1, 32), "nodes": rng.choice([1, 1, 2, 5, 8, 16, spread(rng, 1, 64)]),
             "T": 0, "k": rng.choice([0, 2048, spread(rng, 1, 2048)]),
             "heads": rng.choice([128, 128, 64, 16, rng.randint(1, 128)]), "page": page, "tree": rng.random() < 0.7}
        c["T"] = spread(rng, max(c["nodes"], 2), 200000 if c["k"] else 65536)
        keys = min(c["k"], c["T"]) if c["k"] else c["T"]
        whole = c["B"] * c["nodes"] * keys
        if c["B"] * c["T"] <= 1600000 and whole * c["heads"] <= 8 * 16 * 8192 * 128 and (c["k"] == 0 or whole <= 262144):
            return c


# ---------------------------------------------------------------- inputs
def lengths(case):
    """The sequences' lengths: the first is the longest, the others anywhere from an eighth of it."""
    r = random.Random("%(B)d %(T)d %(nodes)d" % case)
    low = max(case["nodes"], case["T"] // 8)
    return [case["T"]] + [r.randint(low, case["T"]) for _ in range(case["B"] - 1)]


def values(n, width, g):
    """Activations: a size of its own for each token, a few large tokens, a few that are all zero."""
    x = torch.randn(n, width, device="cuda", generator=g)
    u = torch.rand(n, 1, device="cuda", generator=g)
    size = torch.exp(0.3 * torch.randn(n, 1, device="cuda", generator=g))
    return x * torch.where(u < 0.002, 4 * size, torch.where(u > 0.999, 0 * size, size))


def filled(rows, g):
    """Caches in which every row holds a token: rows, their scales, indexer keys, theirs."""
    cache = torch.empty(rows, ROW, dtype=torch.uint8, device="cuda")
    codes = torch.empty(rows, KEYS, dtype=torch.uint8, device="cuda")
    row_scales, key_scales = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    for i in range(0, rows, 1 << 18):
        at = slice(i, min(rows, i + (1 << 18)))
        x = values(at.stop - i, WIDTH + KEYS, g)
        cache[at], row_scales[at] = row_bytes(x[:, :WIDTH])
        c, key_scales[at] = quantised(x[:, WIDTH:])
        codes[at] = c.view(torch.uint8)
    return cache, row_scales, codes, key_scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "attend":
        return prepare_attend(case, seed, g)
    n, rows, dt = case["n"], case["rows"], TYPES[case["dtype"]]
    perm = torch.randperm(rows // 128, device="cuda", generator=g)
    slots = (perm[:, None] * 128 + torch.arange(128, device="cuda")).reshape(-1)[:n].to(torch.int32)
    if case["pad"]:  # every so many-th row of the batch is padding
        slots[case["pad"] - 1::case["pad"]] = -1
    st = {"op": case["op"], "slots": slots, "latent": case["what"] != "index", "index": case["what"] != "latent"}
    if case["op"] == "write":
        # the projection gives latent and indexer key side by side
        x = values(n, WIDTH + KEYS, g).to(dt)
        st["kv"], st["k_idx"] = x[:, :WIDTH], x[:, WIDTH:]
        st["cache"] = torch.zeros(rows, ROW, dtype=torch.uint8, device="cuda")
        st["scales"] = torch.zeros(rows, device="cuda")
        st["keys"] = torch.zeros(rows, KEYS, dtype=torch.uint8, device="cuda")
        st["key_scales"] = torch.zeros(rows, device="cuda")
        st["out"] = {}
        if st["latent"]:
            st["out"].update(codes=st["cache"][:, :VALUES].view(torch.float8_e4m3fn),
                             rest=st["cache"][:, VALUES:].view(torch.bfloat16), scales=st["scales"])
        if st["index"]:
            st["out"].update(key_codes=st["keys"].view(torch.float8_e4m3fn), key_scales=st["key_scales"])
    else:
        st["cache"], st["scales"], st["keys"], st["key_scales"] = filled(rows, g)
        st["out"] = {}
        if st["latent"]:
            st["out"]["kv"] = torch.zeros(n, WIDTH, dtype=dt, device="cuda")
        if st["index"]:
            st["out"]["k_idx"] = torch.zeros(n, KEYS, dtype=dt, device="cuda")
    return st


def prepare_attend(case, seed, g):
    B, L, T, k, heads, page = (case[n] for n in ("B", "nodes", "T", "k", "heads", "page"))
    lens = torch.tensor(lengths(case), dtype=torch.int32)
    pages = (lens + page - 1) // page
    total = int(pages.sum())
    cpu = torch.Generator().manual_seed(seed)
    perm = torch.randperm(total, generator=cpu).to(torch.int32)
    table = torch.full((B, -(-T // page)), -1, dtype=torch.int32)
    table[torch.arange(table.shape[1])[None, :] < pages[:, None]] = perm
    r = random.Random(seed)
    masks = []
    for _ in range(B):
        row = [1]
        for i in range(1, L):  # a node sees itself and what its parent sees
            row.append(1 << i | row[r.randrange(max(0, i - 6), i) if case["tree"] else i - 1])
        masks.append([m - (1 << 64) if m >> 63 else m for m in row])
    st = {"op": "attend", "page": page, "T": T, "scale": WIDTH ** -0.5, "idx": None,
          "lens": lens.cuda(), "table": table.cuda(),
          "tree": torch.tensor(masks, dtype=torch.int64, device="cuda"),
          "q": torch.randn(B, L, heads, WIDTH, device="cuda", generator=g).bfloat16(),
          "out": torch.empty(B, L, heads, VALUES, dtype=torch.bfloat16, device="cuda")}
    st["cache"], st["scales"] = filled(total * page, g)[:2]
    if k:  # positions 0..t of each node, in ascending order, then -1
        t = st["lens"][:, None, None] - L + torch.arange(L, device="cuda")[None, :, None]
        lot = torch.rand(B, L, T, device="cuda", generator=g)
        lot = torch.where(torch.arange(T, device="cuda") <= t, lot, -1.0)
        top, at = lot.topk(min(k, T), dim=-1)
        idx = torch.where(top >= 0, at, T).sort(dim=-1).values
        idx = torch.where(idx < T, idx, -1).to(torch.int32)
        st["idx"] = torch.nn.functional.pad(idx, (0, k - idx.shape[-1]), value=-1).contiguous()
    return st


# ---------------------------------------------------------------- the plain forms
def quantised(x):
    """e4m3 codes of rows and their power-of-two scales."""
    x = x.float()
    top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1, keepdim=True)
    part, e = torch.frexp(top)  # top = part * 2^e, part in [1/2, 1); 448 = 7/8 * 2^9
    e = (e - 9 + (part > 0.875)).clamp(min=-32)
    e = torch.where(top > 0, e, 0).to(torch.int32)
    scale, over = ((e + 127) << 23).view(torch.float32), ((127 - e) << 23).view(torch.float32)
    return (x * over).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale.squeeze(-1)


def row_bytes(kv):
    codes, scales = quantised(kv[:, :VALUES])
    rest = (kv[:, VALUES:].float() / scales[:, None]).to(torch.bfloat16)
    return torch.cat([codes.view(torch.uint8), rest.view(torch.uint8)], -1), scales


def decoded(rows, scales):
    """float32 [..., 576] of cache rows [..., 640]."""
    codes = rows[..., :VALUES].view(torch.float8_e4m3fn).float()
    return torch.cat([codes, rows[..., VALUES:].view(torch.bfloat16).float()], -1) * scales.unsqueeze(-1)


def plain_write(st):
    there = st["slots"] >= 0
    at = st["slots"][there].long()
    if st["latent"]:
        st["cache"][at], st["scales"][at] = row_bytes(st["kv"][there])
    if st["index"]:
        codes, st["key_scales"][at] = quantised(st["k_idx"][there])
        st["keys"][at] = codes.view(torch.uint8)
    return st["out"]


def plain_read(st):
    there, at = (st["slots"] >= 0)[:, None], st["slots"].clamp(min=0).long()
    if st["latent"]:
        st["out"]["kv"].copy_(torch.where(there, decoded(st["cache"][at], st["scales"][at]), 0.0))
    if st["index"]:
        x = st["keys"][at].view(torch.float8_e4m3fn).float() * st["key_scales"][at][:, None]
        st["out"]["k_idx"].copy_(torch.where(there, x, 0.0))
    return st["out"]


def plain_attend(st):
    q, page, lens = st["q"].float(), st["page"], st["lens"][:, None, None]
    B, L, heads, _ = q.shape
    at = torch.arange(st["T"], device=q.device)[None, None] if st["idx"] is None else st["idx"].long()
    node = at - (lens - L)
    bit = (st["tree"][:, :, None] >> node.clamp(0, 63)) & 1
    seen = (at >= 0) & (at < lens) & ((node < 0) | (bit == 1))  # [B, L, keys]
    safe = torch.where((at >= 0) & (at < lens), at, 0)
    row = torch.gather(st["table"].long(), 1, (safe // page).flatten(1)).view(safe.shape) * page + safe % page
    kv = decoded(st["cache"][row], st["scales"][row])  # [B, 1 or L, keys, 576]
    if st["idx"] is None:
        s = torch.matmul(q.flatten(1, 2), kv[:, 0].transpose(1, 2)).view(B, L, heads, -1)
    else:
        s = torch.matmul(q, kv.transpose(2, 3))
    s = torch.where(seen[:, :, None], s * st["scale"], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    v = kv[..., :VALUES]
    o = torch.matmul(p.flatten(1, 2), v[:, 0]).view(B, L, heads, -1) if st["idx"] is None else torch.matmul(p, v)
    st["out"].copy_(torch.where(total > 0, o / total, 0.0))
    return st["out"]


# ---------------------------------------------------------------- one pass
def run(st):
    if own:
        return own_run(st)
    return {"write": plain_write, "read": plain_read, "attend": plain_attend}[st["op"]](st)


def own_run(st):
    import cross_layer_top_full_b200 as ic
    if "ws" not in st:  # the workspace and the batch's description, kept by a program for all its steps
        size = ic.STATUS_BYTES
        if st["op"] == "attend":
            st["pr"] = ic.paged_rows(st["lens"], st["table"], st["T"], st["page"], len(st["cache"]) // st["page"], st["q"].shape[1])
            size = ic.tree_attn_q8_workspace_size(st["pr"], 0 if st["idx"] is None else st["idx"].shape[-1], st["q"].shape[2])
        st["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        ic.workspace_init(st["ws"])
    if st["op"] == "attend":
        ic.tree_attn_q8_paged(st["q"], st["cache"], st["scales"], st["idx"], st["pr"], st["scale"], st["out"], st["ws"], tree=st["tree"])
        return st["out"]
    pick = {}
    if st["op"] == "write":
        if st["latent"]:
            pick.update(kv=st["kv"], kv_q8=st["cache"], kv_scale=st["scales"])
        if st["index"]:
            pick.update(k_idx=st["k_idx"], k_codes=st["keys"], k_scale=st["key_scales"])
        ic.cache_write_q8(st["slots"], st["ws"], **pick)
    else:
        if st["latent"]:
            pick.update(kv=st["out"]["kv"], kv_q8=st["cache"], kv_scale=st["scales"])
        if st["index"]:
            pick.update(k_idx=st["out"]["k_idx"], k_codes=st["keys"], k_scale=st["key_scales"])
        ic.cache_read_q8(st["slots"], st["ws"], **pick)
    return st["out"]


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] != "attend":
        n = case["n"] - (case["n"] // case["pad"] if case["pad"] else 0)
        size = {"bf16": 2, "f32": 4}[case["dtype"]]
        latent, index = case["what"] != "index", case["what"] != "latent"
        there = (WIDTH * size + ROW + 4 if latent else 0) + (KEYS * size + KEYS + 4 if index else 0)
        padded = (WIDTH * size if latent else 0) + (KEYS * size if index else 0) if case["op"] == "read" else 0
        return {"bytes": n * there + (case["n"] - n) * padded + 4 * case["n"], "flops": 0}
    L, k, heads = case["nodes"], case["k"], case["heads"]
    pairs = rows = 0.0
    for T in lengths(case):
        context = T - L
        if k:  # the union of the nodes' random lists
            pairs += sum(min(k, context + i + 1) for i in range(L))
            rows += T * (1 - math.prod(1 - min(k, context + i + 1) / T for i in range(L)))
        else:
            pairs += L * context + L * (L + 1) / 2
            rows += T
    queries = case["B"] * L
    return {"bytes": rows * (ROW + 4) + queries * (heads * (WIDTH + VALUES) * 2 + 4 * k + 8),
            "flops": 2.0 * pairs * heads * (WIDTH + VALUES)}


# ---------------------------------------------------------------- the definition in 64 bits
def two_to(e):
    """2^e of whole numbers e, exactly (pow may be a step off)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def grid(y):
    """The e4m3 number nearest to y, ties to the even one: four significant bits, no step under 2^-9, 448 at most."""
    _, e = torch.frexp(torch.where(y == 0, 1.0, y))
    step = two_to((e - 1).clamp(min=-6) - 3)
    return torch.clamp(torch.round(y / step) * step, -448.0, 448.0)


def row_scale(y):
    top = y.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 448.0) / 448.0))
    e = torch.where(top > 448.0 * two_to(e), e + 1, e)  # what log2 may round at a border
    e = torch.where(top <= 448.0 * two_to(e - 1), e - 1, e)
    return torch.where(top > 0, two_to(e.clamp(min=-32.0)), 1.0)


def numbers(cache, scales):
    """float64 [R, 576] of cache rows."""
    return torch.cat([cache[:, :VALUES].view(torch.float8_e4m3fn).double(),
                      cache[:, VALUES:].view(torch.bfloat16).double()], 1) * scales[:, None].double()


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attend":
        return exact_attend(st)
    slots = st["slots"].long()
    keep = torch.nonzero(slots >= 0).flatten()
    if case["op"] == "read":
        out = {}
        if st["latent"]:
            out["kv"] = torch.zeros(len(slots), WIDTH, dtype=torch.float64, device="cuda")
            out["kv"][keep] = numbers(st["cache"][slots[keep]], st["scales"][slots[keep]])
        if st["index"]:
            out["k_idx"] = torch.zeros(len(slots), KEYS, dtype=torch.float64, device="cuda")
            out["k_idx"][keep] = st["keys"][slots[keep]].view(torch.float8_e4m3fn).double() * st["key_scales"][slots[keep], None].double()
        return out
    rows, out = case["rows"], {}
    zeros = lambda w: torch.zeros(rows, w, dtype=torch.float64, device="cuda")  # noqa: E731
    if st["latent"]:
        out.update(codes=zeros(VALUES), rest=zeros(64), scales=zeros(1)[:, 0])
        x = st["kv"][keep].double()
        y = x[:, :VALUES]
        out["codes"][slots[keep]] = grid(y / row_scale(y))
        out["scales"][slots[keep]] = row_scale(y)[:, 0]
        out["rest"][slots[keep]] = x[:, VALUES:] / row_scale(y)
    if st["index"]:
        out.update(key_codes=zeros(KEYS), key_scales=zeros(1)[:, 0])
        y = st["k_idx"][keep].double()
        out["key_codes"][slots[keep]] = grid(y / row_scale(y))
        out["key_scales"][slots[keep]] = row_scale(y)[:, 0]
    return out


def exact_attend(st):
    B, L, heads, _ = st["q"].shape
    out = torch.zeros(B, L, heads, VALUES, dtype=torch.float64, device="cuda")
    for b in range(B):
        T = int(st["lens"][b])
        pos = torch.arange(T, device="cuda")
        row = st["table"][b].long()[pos // st["page"]] * st["page"] + pos % st["page"]
        dense = numbers(st["cache"][row], st["scales"][row]) if st["idx"] is None else None
        for i in range(L):
            mask = int(st["tree"][b, i])
            seen = torch.tensor([True] * (T - L) + [bool(mask >> a & 1) for a in range(L)], device="cuda")
            if dense is None:
                mine = st["idx"][b, i].long()
                mine = mine[(mine >= 0) & (mine < T)]
                mine = mine[seen[mine]]
                kv = numbers(st["cache"][row[mine]], st["scales"][row[mine]])
            else:
                kv = dense[seen]
            if len(kv):
                p = torch.softmax(st["q"][b, i].double() @ kv.T * st["scale"], -1)
                out[b, i] = p @ kv[:, :VALUES]
    return out
