"""Workloads of the 4-bit paged key/value cache: the plan of a step (block tables and slot maps),
the store (rotary embedding, learned scales, per (token, head) quantization into the pages, and
the read-back of what was stored) and the attention over the cache, for decoding and for prefill.

The cache pool is one uint8 tensor [pages, kv heads, page / 16, 16 D + 256]: a cell holds 16
tokens of one kv head as K codes [16, D / 2], V codes [16, D / 2] (element d of a row in byte
d / 2, low nibble first), then K h [16] float32, K z [16] int32, V h [16] float32, V z [16] int32.
A stored value is (c - z) h with h = max((max - min) / 15, 1e-8), z = -rint(min / h) and
c = clamp(rint(x / h) + z, 0, 15) over the row of D values, in binary32.
"""
import math

import torch

own = False

CELL = 16
H_FLOOR = 1e-8
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # One decoding step of a small server: 8 running requests take one token each.
        dict(name="plan_decode_8", op="plan", requests=8, new=1, longest=2048, page=16, pages=2048),
        # One step of continuous batching: 256 requests, most decoding, every eighth bringing a
        # prompt, some finished and released.
        dict(name="plan_mixed_256", op="plan", requests=256, new=1024, longest=8192, page=32,
             pages=98304),
        # The 7B attention's one new token (32 heads of 128), float32 as the folded q|k|v
        # product leaves it: the smallest store.
        dict(name="store_1_mha", op="store", tokens=1, kv_heads=32, group=1, dim=128, page=16,
             dtype="f32", abits=16, affine=True),
        # A decoding batch of 200 requests, grouped-query heads, bfloat16 projections.
        dict(name="store_200_gqa", op="store", tokens=200, kv_heads=8, group=4, dim=128, page=64,
             dtype="bf16", abits=16, affine=False),
        # The calibration length, 2048 tokens of the 7B block, with the learned scales and the
        # 4-bit queries of W4A4.
        dict(name="store_2048_w4a4", op="store", tokens=2048, kv_heads=32, group=1, dim=128,
             page=64, dtype="f32", abits=4, affine=True),
        # One user decoding at the end of a 2048-token context, 32 heads without grouping.
        dict(name="decode_1x2049", op="attend", requests=1, longest=2049, ragged=False, new=1,
             kv_heads=32, group=1, dim=128, page=16, dtype="f16", causal=True),
        # A busy server's decoding step: 64 ragged contexts of up to 8192 tokens.
        dict(name="decode_64x8192", op="attend", requests=64, longest=8192, ragged=True, new=1,
             kv_heads=8, group=4, dim=128, page=64, dtype="bf16", causal=True),
        # One request at a very long context: few rows, one long axis.
        dict(name="decode_1x131072", op="attend", requests=1, longest=131072, ragged=False, new=1,
             kv_heads=8, group=4, dim=128, page=64, dtype="bf16", causal=True),
        # Checking five drafted tokens for 33 requests, heads of 64.
        dict(name="verify_33x4001x5", op="attend", requests=33, longest=4001, ragged=True, new=5,
             kv_heads=4, group=2, dim=64, page=32, dtype="f16", causal=True),
        # The prompt of one 2048-token calibration sample through the 7B attention.
        dict(name="prefill_2048_mha", op="attend", requests=1, longest=2048, ragged=False, new=2048,
             kv_heads=32, group=1, dim=128, page=16, dtype="bf16", causal=True),
        # Chunked prefill: three ragged chunks of up to 1000 tokens behind contexts of up to 16k.
        dict(name="chunk_3x1000_16k", op="attend", requests=3, longest=16411, ragged=True, new=1000,
             kv_heads=8, group=4, dim=128, page=64, dtype="bf16", causal=True),
        # A long prompt at once: the largest product.
        dict(name="prefill_8192", op="attend", requests=1, longest=8192, ragged=False, new=8192,
             kv_heads=8, group=4, dim=128, page=128, dtype="bf16", causal=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


MOST_ROWS = 64 * 8192 * 8 * 128           # cached values of one kind, padded to the longest
MOST_PAIRS = 32 * 8192 * 4096             # (query head, query, key) triples


def draw(rng):
    op = rng.choice(["plan", "store", "store", "attend", "attend", "attend"])
    if op == "plan":
        page = rng.choice([16, 32, 64, 128])
        case = dict(op=op, requests=_log_int(rng, 1, 256), new=_log_int(rng, 1, 1024),
                    longest=_log_int(rng, 64, 8192), page=page)
        lens, new = _plan_sizes(case)
        held = sum(-(-a // page) for a in lens)
        need = sum(-(-(a + b) // page) for a, b in zip(lens, new) if b > 0) - held
        # from a pool that refuses some requests to one with room to spare
        case["pages"] = max(1, held + int(max(0, need) * rng.choice([0.5, 1.0, 3.0])))
        return case
    dim = rng.choice([64, 128, 128])
    kv_heads, group = rng.choice([(1, 8), (2, 4), (4, 2), (4, 7), (8, 1), (8, 4), (8, 8), (32, 1)])
    page = rng.choice([16, 32, 64, 128])
    if op == "store":
        return dict(op=op, tokens=_log_int(rng, 1, 2048), kv_heads=kv_heads, group=group, dim=dim,
                    page=page, dtype=rng.choice(["f32", "bf16", "f16"]),
                    abits=rng.choice([16, 16, 4, 8]), affine=rng.random() < 0.5)
    requests = _log_int(rng, 1, 64)
    longest = _log_int(rng, 1, 131072)
    while requests * longest * kv_heads * dim > MOST_ROWS:
        longest = max(1, longest // 2)
    kind = rng.choice(["decode", "verify", "prefill"])
    new = 1 if kind == "decode" else rng.randint(2, 8) if kind == "verify" else _log_int(rng, 9, 4096)
    new = min(new, longest)
    while requests * new * longest * kv_heads * group > MOST_PAIRS:
        new = max(1, new // 2)
    return dict(op=op, requests=requests, longest=longest, ragged=rng.random() < 0.7, new=new,
                kv_heads=kv_heads, group=group, dim=dim, page=page,
                dtype=rng.choice(["bf16", "f16"]), causal=new == 1 or rng.random() < 0.9)


def _spread(case, n, lo, hi):
    """n whole numbers over lo .. hi, evenly by the golden ratio, the first of them hi."""
    return [hi - int((i * 0.6180339887498949 % 1.0) * (hi - lo + 1)) for i in range(n)]


def _requests(case):
    """(lengths with the new tokens, new tokens) of an attention case."""
    n, L = case["requests"], case["longest"]
    if not case["ragged"]:
        return [L] * n, [case["new"]] * n
    lens = _spread(case, n, max(1, L // 16), L)
    new = _spread(case, n, max(1, case["new"] // 2), case["new"]) if case["new"] > 8 else \
        [case["new"]] * n
    return lens, [min(a, b) for a, b in zip(new, lens)]


def _plan_sizes(case):
    """(lengths, new tokens) of a plan case: decoding, prompts, released requests."""
    n = case["requests"]
    lens = _spread(case, n, 0, case["longest"])
    if case["new"] == 1:
        return lens, [1] * n
    prompts = _spread(case, n, 2, case["new"])
    new = [prompts[i] if i % 8 == 3 else -1 if i % 16 == 5 else 1 for i in range(n)]
    return lens, new


def work(case):
    if case["op"] == "plan":
        lens, new = _plan_sizes(case)
        tokens = sum(max(0, x) for x in new)
        pages = sum(-(-(a + b) // case["page"]) + (a // -case["page"]) for a, b in zip(lens, new) if b > 0)
        return {"bytes": 4 * (3 * len(lens) + 2 + 2 * pages) + 12 * tokens, "flops": 0}
    d, hk = case["dim"], case["kv_heads"]
    hq = hk * case["group"]
    if case["op"] == "store":
        size = 4 if case["dtype"] == "f32" else 2
        t = case["tokens"]
        return {"bytes": t * ((hq + 2 * hk) * d * size + hq * d * 2 + 2 * hk * (d + 16)
                              + 2 * hk * d * 4 + 4 * d + 8), "flops": 0}
    lens, new = _requests(case)
    pairs = 0
    for a, n in zip(lens, new):
        pairs += n * (a - n) + n * (n + 1) // 2 if case["causal"] else n * a
    kv = sum(lens) * hk * (d + 16)
    return {"bytes": kv + 4 * sum(new) * hq * d + sum(-(-a // case["page"]) for a in lens) * 4,
            "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------------------ the inputs

def _quantize(x, levels=15.0):
    """(codes, h, z) of the rows of x (float32), in binary32 with one rounding per operation."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    h = (hi - lo) / torch.full_like(hi, levels)       # by a tensor: a true quotient
    h = torch.where(h >= H_FLOOR, h, torch.full_like(h, H_FLOOR))
    z = -torch.round(lo / h)
    return torch.clamp(torch.round(x / h) + z, 0.0, levels), h, z


def _parts(pool, dim):
    """Views of a pool: K codes, V codes [.., 16, D / 2]; K h, K z, V h, V z [.., 16]."""
    half = CELL * dim // 2
    shape = pool.shape[:3]
    codes = [pool[..., i * half:(i + 1) * half].view(*shape, CELL, dim // 2) for i in range(2)]
    at = 2 * half
    meta = [pool[..., at + 64 * i: at + 64 * (i + 1)].view(t) for i, t in
            enumerate((torch.float32, torch.int32, torch.float32, torch.int32))]
    return codes + meta


def _pack(c):
    c = c.to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _unpack(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2).float()


def _filled_pool(gen, pages, case):
    """A pool whose every slot holds a quantized row: what earlier steps left there."""
    hk, d, cells = case["kv_heads"], case["dim"], case["page"] // CELL
    pool = torch.empty(pages, hk, cells, CELL * d + 256, dtype=torch.uint8, device="cuda")
    kc, vc, kh, kz, vh, vz = _parts(pool, d)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    # keys have channels of a large mean and of a large spread, values are milder
    spread = torch.exp(0.4 * r(hk, 1, 1, d))
    for codes, h, z, scale, shift in ((kc, kh, kz, spread, 0.7 * r(hk, 1, 1, d)),
                                      (vc, vh, vz, 0.5, 0.1 * r(hk, 1, 1, d))):
        c, hh, zz = _quantize(r(pages, hk, cells, CELL, d) * scale + shift)
        codes.copy_(_pack(c))
        h.copy_(hh[..., 0])
        z.copy_(zz[..., 0])
        del c, hh, zz
    return pool


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prefix(values):
    out = [0]
    for v in values:
        out.append(out[-1] + v)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=dict(case))
    if case["op"] == "plan":
        lens, new = _plan_sizes(case)
        page, n = case["page"], case["requests"]
        order = torch.randperm(n, generator=gen, device="cuda")
        s["lens"], s["new"] = _ints(lens)[order], _ints(new)[order]
        width = -(-(case["longest"] + case["new"]) // page)
        held = (s["lens"].long() + page - 1) // page
        col = torch.arange(width, device="cuda")
        used = col[None, :] < held[:, None]
        ids = torch.randperm(case["pages"], generator=gen, device="cuda").int()
        at = used.flatten().cumsum(0).view(n, width) - 1
        s["table"] = torch.where(used, ids[at.clamp(min=0)], -1)
        taken = sum(-(-a // page) for a in lens)
        s["free"] = torch.cat((ids[taken:], ids[:taken]))
        s["n_free"] = _ints([case["pages"] - taken])
        s["capacity"] = sum(max(0, x) for x in new)
        return s
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    hq = hk * case["group"]
    dt = DTYPES[case["dtype"]]
    r = lambda *sh: torch.randn(*sh, generator=gen, device="cuda")  # noqa: E731
    if case["op"] == "store":
        t = case["tokens"]
        qkv = r(t, (hq + 2 * hk) * d) * torch.exp(0.5 * r((hq + 2 * hk) * d))
        qkv = qkv.to(dt)
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        s["v"] = qkv[:, (hq + hk) * d:].unflatten(1, (hk, d))
        pages = -(-t // page) + 7
        s["pool"] = _filled_pool(gen, pages, case)
        # the tokens' slots, page after page of a shuffled table; positions behind a context
        order = torch.randperm(pages, generator=gen, device="cuda")
        i = torch.arange(t, device="cuda")
        s["slots"] = (order[i // page] * page + i % page).int()
        first = int(torch.randint(0, 2048, (1,), generator=gen, device="cuda"))
        s["positions"] = (first + i).int()
        angle = torch.arange(4096, device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(d // 2, device="cuda", dtype=torch.float64) * 2 / d)
        s["rope"] = torch.stack((angle.cos(), angle.sin())).float()
        if case["affine"]:
            s["s_a"], s["s_o"] = torch.exp(0.3 * r(hk, d)), torch.exp(0.3 * r(hk, d))
            s["delta_o"] = 0.2 * r(hk, d)
        else:
            s["s_a"] = s["s_o"] = s["delta_o"] = None
        return s
    lens, new = _requests(case)
    need = [-(-a // page) for a in lens]
    width, total = max(need), sum(need)
    s["pool"] = _filled_pool(gen, total + 3, case)
    ids = torch.randperm(total + 3, generator=gen, device="cuda").int()
    col = torch.arange(width, device="cuda")
    used = col[None, :] < _ints(need)[:, None]
    at = used.flatten().cumsum(0).view(len(need), width) - 1
    s["table"] = torch.where(used, ids[at.clamp(min=0)], -1)
    s["lens"], s["cu"] = _ints(lens), _ints(_prefix(new))
    s["q"] = r(sum(new), hq, d).to(dt)
    s["max_q"] = max(new)
    return s


# ------------------------------------------------------------------------------ plain forms

def _plan_plain(s):
    case = s["case"]
    page, pages, cap = case["page"], case["pages"], s["capacity"]
    lens, table = s["lens"].long(), s["table"]
    n_req, width = table.shape
    release = s["new"] < 0
    new = s["new"].long().clamp(min=0)
    held, after = (lens + page - 1) // page, (lens + new + page - 1) // page
    wide = after > width
    need = torch.where(release | wide, 0, after - held)
    new = torch.where(wide, 0, new)
    col = torch.arange(width, device=lens.device)
    # pages that come back go on top of the stack
    back = release[:, None] & (col[None, :] < held[:, None])
    to = s["n_free"].long() + back.flatten().cumsum(0) - 1
    free = torch.cat((s["free"], s["free"].new_zeros(1)))
    free = free.scatter(0, torch.where(back.flatten(), to, pages), table.flatten())[:pages]
    avail = s["n_free"].long() + back.sum()
    # who fits, in request order
    pre = need.cumsum(0)
    ok = (need == 0) | (pre <= avail)
    new = torch.where(ok, new, 0)
    ok = ok & ((new == 0) | (new.cumsum(0) <= cap))
    new, need = torch.where(ok, new, 0), torch.where(ok, need, 0)
    cu = torch.cat((new.new_zeros(1), new.cumsum(0)))
    at = col[None, :] - held[:, None]
    fresh = (at >= 0) & (at < need[:, None])
    pop = avail - 1 - ((pre - need)[:, None] + at)
    table = torch.where(fresh, free[pop.clamp(0, pages - 1)], table)
    # the tokens' request, position and slot
    i = torch.arange(cap, device=lens.device)
    req = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    live = i < cu[-1]
    req = req.clamp(max=n_req - 1)
    pos = lens[req] + i - cu[req]
    at = (pos // page).clamp(0, width - 1)
    slot = table[req, at].long() * page + pos % page
    out = lambda x: torch.where(live, x, -1).int()  # noqa: E731
    lens = torch.where(release, 0, lens + new).int()
    return dict(lens=lens, n_free=(avail - need.sum()).int(), cu=cu.int(), slots=out(slot),
                positions=out(pos), requests=out(req), table=table, free=free)


def _rope(x, cs):
    half = x.shape[-1] // 2
    a, b = x[..., :half], x[..., half:]
    c, s = cs[0][:, None], cs[1][:, None]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _store_plain(s):
    case = s["case"]
    d, page = case["dim"], case["page"]
    cs = s["rope"][:, s["positions"].long()]
    q, k, v = _rope(s["q"].float(), cs), _rope(s["k"].float(), cs), s["v"].float()
    if s["s_a"] is not None:
        q = q / s["s_a"].repeat_interleave(case["group"], 0)
        k = k * s["s_a"]
        v = (v - s["delta_o"]) / s["s_o"]
    if case["abits"] < 16:
        c, h, z = _quantize(q, float(2 ** case["abits"] - 1))
        q = (c - z) * h
    slot = s["slots"].long()
    at = (slot // page, slice(None), slot % page // CELL, slot % CELL)
    parts = _parts(s["pool"], d)
    read = []
    for x, (codes, h, z) in ((k, (parts[0], parts[2], parts[3])), (v, (parts[1], parts[4], parts[5]))):
        c, hh, zz = _quantize(x)
        codes[at], h[at], z[at] = _pack(c), hh[..., 0], zz[..., 0].int()
        read.append((_unpack(codes[at]) - z[at].float()[..., None]) * h[at][..., None])
    return dict(q=q.to(torch.float16), k=read[0], v=read[1])


def _attend_plain(s):
    case = s["case"]
    d, hk, g = case["dim"], case["kv_heads"], case["group"]
    n_req, n = s["lens"].numel(), s["max_q"]
    kc, vc, kh, kz, vh, vz = _parts(s["pool"], d)
    ids = s["table"].clamp(min=0).long()
    value = lambda c, h, z: ((_unpack(c[ids]) - z[ids].float()[..., None]) * h[ids][..., None]) \
        .transpose(1, 2).reshape(n_req, hk, -1, d)  # noqa: E731
    k, v = value(kc, kh, kz), value(vc, vh, vz)
    first, count = s["cu"][:-1].long(), s["cu"][1:].long() - s["cu"][:-1].long()
    i = torch.arange(n, device=first.device)
    rows = (first[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[rows].view(n_req, n, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n_req, hk, g * n, d)
    x = (q @ k.transpose(2, 3)) * d ** -0.5
    x = x.view(n_req, hk, g, n, -1)
    j = torch.arange(x.shape[-1], device=first.device)
    last = s["lens"].long()[:, None] - 1
    if case["causal"]:
        last = (s["lens"].long() - count)[:, None] + i
    else:
        last = last.expand(n_req, n)
    seen = (j <= last[:, :, None]) & (j < s["lens"][:, None, None])
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(torch.isfinite(top), top, 0.0)).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(n_req, hk, g * n, -1) @ v).view(n_req, hk, g, n, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(n_req, n, hk * g, d)
    t = torch.arange(s["q"].shape[0], device=first.device)
    req = torch.searchsorted(s["cu"][1:].long().contiguous(), t, right=True)
    return o[req, t - first[req]].to(s["q"].dtype)


def run(state):
    case = state["case"]
    if own:
        from post_quantization_lwc_b200 import omq
        if case["op"] == "plan":
            p = omq.kv_plan(state["lens"], state["new"], state["table"], state["free"],
                            state["n_free"], case["page"], state["capacity"])
            return dict(lens=p["lens"], n_free=p["n_free"], cu=p["cu"], slots=p["slots"],
                        positions=p["positions"], requests=p["requests"], table=state["table"],
                        free=state["free"])
        if case["op"] == "store":
            q = omq.kv_append(state["pool"], state["slots"], state["k"], state["v"], q=state["q"],
                              positions=state["positions"], rope=state["rope"],
                              s_a=state["s_a"], s_o=state["s_o"], delta_o=state["delta_o"],
                              abits=case["abits"], q_dtype=torch.float16)
            k, v = omq.kv_read(state["pool"], state["slots"], dtype=torch.float32)
            return dict(q=q, k=k, v=v)
        return omq.kv_attn(state["q"], state["pool"], state["table"], state["lens"], state["cu"],
                           state["max_q"], causal=case["causal"])
    if case["op"] == "plan":
        return _plan_plain(state)
    if case["op"] == "store":
        return _store_plain(state)
    return _attend_plain(state)


# ------------------------------------------------------------------------------ 64 bits

def _exact_rows(x, top):
    """The stored values of the rows of x. The encoder's integers are defined by binary32
    operations (numpy's, one rounding each); the values they stand for are taken in 64 bits."""
    import numpy as np
    f = np.float32
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    h = np.maximum(((hi - lo).astype(f) / f(top)).astype(f), f(H_FLOOR))
    z = -np.rint((lo / h).astype(f))
    c = np.clip(np.rint((x / h).astype(f)) + z, f(0), f(top))
    return (c.astype(np.float64) - z.astype(np.float64)) * h.astype(np.float64)


def _exact_store(case, s):
    import numpy as np
    host = lambda t: None if t is None else t.float().cpu().numpy()  # noqa: E731
    f, half = np.float32, case["dim"] // 2
    cos, sin = (host(s["rope"])[i][s["positions"].cpu().numpy()][:, None, :] for i in (0, 1))
    turned = []
    for name in ("q", "k"):
        x = host(s[name])
        a, b = x[..., :half], x[..., half:]
        turned.append(np.concatenate(((a * cos).astype(f) - (b * sin).astype(f),
                                      (b * cos).astype(f) + (a * sin).astype(f)), -1))
    q, k = turned
    v = host(s["v"])
    if case["affine"]:
        sa, so, dl = host(s["s_a"]), host(s["s_o"]), host(s["delta_o"])
        q = q / np.repeat(sa, case["group"], axis=0)
        k = k * sa
        v = (v - dl) / so
    q = _exact_rows(q, 2 ** case["abits"] - 1) if case["abits"] < 16 else q.astype(np.float64)
    return dict(q=q, k=_exact_rows(k, 15), v=_exact_rows(v, 15))


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    if case["op"] == "store":
        return _exact_store(case, s)
    d, hk, g, page = case["dim"], case["kv_heads"], case["group"], case["page"]
    lens, cu = s["lens"].tolist(), s["cu"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    half = CELL * d // 2
    for b, n_keys in enumerate(lens):
        n_new = cu[b + 1] - cu[b]
        mine = s["pool"][s["table"][b, : -(-n_keys // page)].long()]
        for head in range(hk):
            cell = mine[:, head].reshape(-1, CELL * d + 256)
            kv = []
            for at, meta in ((0, 2 * half), (half, 2 * half + 128)):
                byte = cell[:, at:at + half].reshape(-1, d // 2)
                c = torch.empty(byte.shape[0], d, dtype=torch.float64, device="cuda")
                c[:, ::2], c[:, 1::2] = byte % 16, byte // 16
                h = cell[:, meta:meta + 64].contiguous().view(torch.float32).reshape(-1, 1)
                z = cell[:, meta + 64:meta + 128].contiguous().view(torch.int32).reshape(-1, 1)
                kv.append(((c - z.double()) * h.double())[:n_keys])
            for j in range(g):
                q = s["q"][cu[b]:cu[b + 1], head * g + j].double()
                x = q @ kv[0].T / math.sqrt(d)
                if case["causal"]:
                    hide = torch.ones(n_new, n_keys, dtype=torch.bool, device="cuda").triu(n_keys - n_new + 1)
                    x.masked_fill_(hide, -math.inf)
                out[cu[b]:cu[b + 1], head * g + j] = torch.softmax(x, -1) @ kv[1]
    return out
