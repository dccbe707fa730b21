"""The operators of a decode step that reads only the pages of a long paged context that matter, as cases
that can be timed and compared.

* ``map``    -- positions and slots of the new tokens, from the batch's lengths and page table;
* ``rope``   -- rotary positions of q and k with the write of K and V into the paged pool;
* ``bound``  -- 8-bit lower and upper bounds of the keys of each page, per KV head and channel;
* ``select`` -- the pages of every (token, KV head) with the largest upper bound of q.k;
* ``attend`` -- decode attention over the selected pages;
* ``step``   -- bound, select and attend, one after the other, as a layer of a decode step calls them.

``run`` computes them in plain torch, in 32 bits (64 where sums are whole numbers or angles are far), or, where
``own`` is true, makes the framework's calls.
"""

import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of the eight E2M1 codes


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # a large batch's decode step: one token per request, launch latency counts
        dict(name="map_step", op="map", batch=256, lo=16, hi=8192, len_seed=1, page=64, new="one"),
        # prompts being extended by chunks beside requests that decode
        dict(name="map_mixed", op="map", batch=64, lo=512, hi=4096, len_seed=2, page=16, new="some"),
        # one decode step of 64 requests at far positions
        dict(name="rope_step", op="rope", tokens=64, heads=32, kv_heads=8, dim=128, rotary=128, interleaved=False, dtype="bf16",
             page=16, base=500000.0, factor=1.0, far=131071),
        # the new tokens of a few prompts, an odd number of them; frequencies scaled for a context eight times as long
        dict(name="rope_prompt", op="rope", tokens=8191, heads=32, kv_heads=8, dim=128, rotary=128, interleaved=False, dtype="bf16",
             page=16, base=500000.0, factor=8.0, far=131071),
        # neighbouring pairs over half of each head, an E4M3 cache scattered token by token
        dict(name="rope_part_e4m3", op="rope", tokens=2047, heads=64, kv_heads=8, dim=128, rotary=64, interleaved=True, dtype="e4m3",
             page=1, base=10000.0, factor=1.0, far=32767),
        # the bounds of the pages that a decode step of 64 chats wrote to
        dict(name="bound_step", op="bound", batch=64, lo=512, hi=4096, len_seed=3, page=16, kv_heads=8, dim=128, dtype="bf16",
             every=False),
        # the bounds of every page of 64 chats, as after their prompts
        dict(name="bound_batch64", op="bound", batch=64, lo=512, hi=4096, len_seed=4, page=16, kv_heads=8, dim=128, dtype="bf16",
             every=True),
        # 64 of up to 256 pages of 64 chats
        dict(name="select_batch64", op="select", batch=64, lo=512, hi=4096, len_seed=5, page=16, heads=32, kv_heads=8, dim=128,
             blocks=64, sink=1, recent=2),
        # 256 of 8192 pages of two long documents: few rows, the work split over the pages
        dict(name="select_long", op="select", batch=2, lo=131071, hi=131071, len_seed=6, page=16, heads=32, kv_heads=8, dim=128,
             blocks=256, sink=1, recent=4),
        # the attention of 64 chats over their 64 pages
        dict(name="attend_batch64", op="attend", batch=64, lo=512, hi=4096, len_seed=7, page=16, heads=32, kv_heads=8, dim=128,
             dtype="bf16", blocks=64, sink=1, recent=2),
        # two long documents in a 4-bit cache of large pages, 64 query heads
        dict(name="attend_long4", op="attend", batch=2, lo=131071, hi=131071, len_seed=8, page=128, heads=64, kv_heads=8, dim=128,
             dtype="nvfp4", blocks=32, sink=1, recent=1),
        # a layer of a decode step of two long documents
        dict(name="step_long", op="step", batch=2, lo=131071, hi=131071, len_seed=9, page=16, heads=32, kv_heads=8, dim=128,
             dtype="bf16", blocks=256, sink=1, recent=4),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["map", "rope", "bound", "select", "attend", "step"])
    if op == "rope":
        heads, kv_heads = rng.choice([(32, 8), (64, 8), (8, 8), (28, 4), (40, 8), (16, 1), (32, 1)])
        dtype = rng.choice(["bf16", "e4m3"])
        dim = rng.choice([64, 128]) if dtype == "bf16" else 128
        return dict(op=op, tokens=_log_int(rng, 1, 8191 * 48 // (heads + 2 * kv_heads)), heads=heads, kv_heads=kv_heads, dim=dim,
                    rotary=rng.choice([16, 32, 48, 64] if dim == 64 else [32, 64, 96, 128]), interleaved=rng.random() < 0.5,
                    dtype=dtype, page=rng.choice([1, 16, 32, 64, 128]), base=rng.choice([10000.0, 500000.0, 1000000.0]),
                    factor=rng.choice([1.0, 4.0, 8.0, 32.0]), far=_log_int(rng, 1, 1 << 20))
    # keys of all requests: at most those of the 64 chats, or of the two long documents
    page = rng.choice([16, 32, 64, 128])
    batch = _log_int(rng, 1, 256)
    hi = _log_int(rng, 1, min(131072, 131072 // batch if op == "bound" else 262144 // batch))
    case = dict(op=op, batch=batch, lo=rng.randint(max(1, hi // 8), hi), hi=hi, len_seed=rng.randrange(1 << 30), page=page)
    if op == "map":
        return dict(case, new=rng.choice(["one", "some", "all"]))
    if op != "select":
        case["dtype"] = rng.choice(["bf16", "e4m3", "nvfp4"])
    case["dim"] = rng.choice([64, 128]) if case.get("dtype", "bf16") == "bf16" else 128
    if op == "bound":
        return dict(case, kv_heads=rng.choice([1, 2, 4, 8]), every=rng.random() < 0.5)
    heads, kv_heads = rng.choice([(32, 8), (64, 8), (8, 8), (28, 4), (40, 8), (16, 1), (32, 1)])
    sink, recent = rng.choice([0, 1, 2]), rng.choice([1, 2, 4])
    most = min(512, 65536 // (batch * page))  # keys that are attended to: at most those of the 64 chats
    if sink + recent >= most:
        sink, recent = 0, 1
    blocks = _log_int(rng, min(most, sink + recent + 1), most)
    if op == "select":  # some pages of every request compete, a few at least
        blocks = max(sink + recent + 1, min(blocks, hi // (2 * page)))
        case["lo"] = max(case["lo"], (blocks + 1) * page)
        case["hi"] = max(case["lo"], hi)
    return dict(case, heads=heads, kv_heads=kv_heads, blocks=blocks, sink=sink, recent=recent)


def _lengths(case):
    """The requests' KV lengths and numbers of new tokens: the case's own, not the seed's."""
    r = np.random.RandomState(case["len_seed"])
    L = r.randint(case["lo"], case["hi"] + 1, case["batch"]).astype(np.int64)
    new = case.get("new", "one")
    if new == "one":
        return L, np.ones_like(L)
    if new == "all":
        return L, L.copy()
    n = np.minimum(L, r.randint(0, 512, case["batch"]))  # some without new tokens, some with one, some with a chunk
    return L, np.where(r.rand(case["batch"]) < 0.5, np.minimum(n, 1), n)


def _row(case):
    """Bytes of one key's (or value's) row of one head."""
    return {"bf16": 2 * case["dim"], "e4m3": case["dim"], "nvfp4": case["dim"] // 2 + case["dim"] // 16}[case["dtype"]]


def work(case):
    if case["op"] == "rope":
        T, D, Hq, H = case["tokens"], case["dim"], case["heads"], case["kv_heads"]
        # q in and out, k and v in, the pool's rows out, a position and a slot
        return {"bytes": T * (Hq * D * 4 + 2 * H * D * 2 + 2 * H * _row(case) + 16), "flops": T * (Hq + H) * case["rotary"] * 3}
    L, n = _lengths(case)
    page = case["page"]
    N = -(-L // page)
    if case["op"] == "map":
        T = int(n.sum())
        return {"bytes": T * 16 + len(L) * 16 + int(np.sum(-(-n // page))) * 4, "flops": T * 4}
    H, D = case["kv_heads"], case["dim"]
    r = {"bytes": 0, "flops": 0}
    if case["op"] in ("bound", "step"):
        # the keys of the pages, and both bounds of each
        every = case.get("every", False)
        keys, pages = (int(L.sum()), int(N.sum())) if every else (int(np.sum((L - 1) % page + 1)), len(L))
        r["bytes"] += keys * H * _row(case) + pages * H * 2 * D + H * D * 4
        r["flops"] += keys * H * D * 2
    if case["op"] in ("select", "step"):
        # the bounds of the pages that compete, the queries, the selection
        over = N[N > case["blocks"]]
        r["bytes"] += int(over.sum()) * (H * 2 * D + 4) + len(L) * (case["heads"] * D * 2 + H * case["blocks"] * 4)
        r["flops"] += int(over.sum()) * H * 4 * D
    if case["op"] in ("attend", "step"):
        keys = int(np.sum((np.minimum(N, case["blocks"]) - 1) * page + (L - 1) % page + 1))
        r["bytes"] += keys * H * 2 * _row(case) + len(L) * case["heads"] * (D * 4 + 4) + len(L) * H * case["blocks"] * 8
        r["flops"] += 4 * keys * case["heads"] * D
    return r


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _to_codes(x, scale):
    """bf16 rows [..., D] as packed E2M1 codes [..., D / 2] and E4M3 scale codes [..., D / 16] (uint8)."""
    t = (x.float() * (1.0 / scale)).unflatten(-1, (-1, 16))
    s = (t.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = s.float().unsqueeze(-1)
    a = torch.where(f > 0, t / torch.where(f > 0, f, torch.ones_like(f)), torch.zeros_like(t))
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.bucketize(a.abs(), edges).to(torch.uint8)
    code = (code + 8 * torch.signbit(a).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], s.view(torch.uint8)


def _pools(case, pages, g):
    """K and V pools of the case's type, N(0, 1) values, and the scale of each tensor."""
    page, H, D = case["page"], case["kv_heads"], case["dim"]
    k = torch.randn((pages, page, H, D), generator=g, device="cuda", dtype=torch.bfloat16)
    v = torch.randn((pages, page, H, D), generator=g, device="cuda", dtype=torch.bfloat16)
    if case["dtype"] == "bf16":
        return dict(k=k, v=v, k_scale=1.0, v_scale=1.0)
    ks, vs = (float(np.float32(float(x.abs().max()) / (448.0 if case["dtype"] == "e4m3" else 448.0 * 6.0))) for x in (k, v))
    if case["dtype"] == "e4m3":
        k, v = ((x.float() * (1.0 / s)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x, s in ((k, ks), (v, vs)))
        return dict(k=k, v=v, k_scale=ks, v_scale=vs)
    p = dict(k_scale=ks, v_scale=vs)
    for n, x, s in (("k", k, ks), ("v", v, vs)):
        # the tokens of one head next to each other in a page
        c, f = _to_codes(x.transpose(1, 2).contiguous(), s)
        p[n], p[n + "_sf"] = c.transpose(1, 2), f.transpose(1, 2)
    return p


def _frequencies(case):
    """Angle per position of each pair, float64: base^(-2 i / R); where the context is scaled, wavelengths beyond a
    quarter of the original 8192 positions grow by the factor, and smoothly from there up to the whole of it."""
    f = case["base"] ** (-np.arange(0, case["rotary"], 2, dtype=np.float64) / case["rotary"])
    if case["factor"] == 1.0:
        return f
    turns = 8192.0 * f / (2 * math.pi)  # over the original context
    part = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
    return (1.0 - part) * f / case["factor"] + part * f


def _rope_state(case, g):
    T, Hq, H, D, page = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    # one projection's output, as a layer has it: q, k and v are views of it
    qkv = torch.randn((T, (Hq + 2 * H) * D), generator=g, device="cuda", dtype=torch.bfloat16)
    q, k, v = qkv.split([Hq * D, H * D, H * D], dim=1)
    pages = -(-T // page) * 5 // 4 + 1
    kind = torch.bfloat16 if case["dtype"] == "bf16" else torch.uint8
    s = dict(case, q=q.unflatten(1, (Hq, D)), kn=k.unflatten(1, (H, D)), vn=v.unflatten(1, (H, D)),
             k=torch.zeros((pages, page, H, D), dtype=kind, device="cuda"), v=torch.zeros((pages, page, H, D), dtype=kind, device="cuda"),
             k_scale=1.0 if kind == torch.bfloat16 else 0.015625, v_scale=1.0 if kind == torch.bfloat16 else 0.01171875,
             slots=torch.randperm(pages * page, generator=g, device="cuda")[:T],
             positions=torch.randint(0, case["far"] + 1, (T,), generator=g, device="cuda"),
             freq=torch.from_numpy(_frequencies(case)).cuda())
    if own:
        import paged_kv_attention_slot_gb300 as pk
        s["cache"] = pk.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["rotary_of"] = pk.Rotary(D, rotary_dim=case["rotary"], base=case["base"], interleaved=case["interleaved"],
                                   **({} if case["factor"] == 1.0 else dict(scaling="wavelength", factor=case["factor"],
                                                                            original_positions=8192, low_turns=1.0, high_turns=4.0)))
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "rope":
        return _rope_state(case, g)
    L, n = _lengths(case)
    page, B = case["page"], len(L)
    need = -(-L // page)
    pages = int(need.sum()) * 5 // 4 + 1
    perm = torch.randperm(pages, generator=g, device="cuda")[:int(need.sum())]
    indptr, qo = (np.concatenate([[0], np.cumsum(x)]) for x in (need, n))
    s = dict(case, L=torch.from_numpy(L).cuda(), n=torch.from_numpy(n).cuda(), most=int(need.max()), T=int(n.sum()),
             indptr=torch.from_numpy(indptr).cuda(), qo=torch.from_numpy(qo).cuda(), pages=perm, num_pages=pages)
    # page of every logical block, [B, most] (page 0 behind a request's end)
    at = s["indptr"][:-1, None] + torch.arange(s["most"], device="cuda")
    inside = at < s["indptr"][1:, None]
    s["table"] = torch.where(inside, perm[torch.where(inside, at, 0)], 0)
    if "dtype" in case:
        s.update(_pools(case, pages, g))
    H, D = case.get("kv_heads", 8), case.get("dim", 128)
    if case["op"] in ("bound", "select", "step"):
        # the bounds of each page as an earlier step left them, and their step sizes by head and channel
        s["scale"] = torch.rand((H, D), generator=g, device="cuda") * 0.03 + 0.03
        middle = torch.randn((pages, H, 1, D), generator=g, device="cuda") * 8
        half = torch.rand((pages, H, 1, D), generator=g, device="cuda") * 32 + 24
        s["codes"] = torch.cat((middle - half, middle + half), 2).round().clamp(-127, 127).to(torch.int8)
    if case["op"] in ("select", "attend", "step"):
        s["q"] = torch.randn((B, case["heads"], D), generator=g, device="cuda", dtype=torch.bfloat16)
    if case["op"] == "attend":
        s["chosen"] = _best(s, torch.rand((B, H, s["most"]), generator=g, device="cuda"))
    if own:
        import paged_kv_attention_slot_gb300 as pk
        if "dtype" in case:
            sf = dict(k_sf=s["k_sf"], v_sf=s["v_sf"]) if case["dtype"] == "nvfp4" else {}
            s["cache"] = pk.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"], **sf)
        if "codes" in s:
            s["bounds"] = pk.KeyBounds(s["codes"], s["scale"])
        s["plan"] = pk.Plan().plan(qo.astype(np.int32), indptr.astype(np.int32), perm.cpu().numpy().astype(np.int32),
                                   (L - (need - 1) * page).astype(np.int32), num_qo_heads=case.get("heads", H), num_kv_heads=H,
                                   head_dim=D, page_size=page, mode="mixed" if case["op"] == "map" else "decode",
                                   kv_dtype=case.get("dtype", "bf16"), num_blocks=case.get("blocks", 0))
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(s):
    return {"map": _map, "rope": _rope, "bound": _bound, "select": _select, "attend": _attend, "step": _step}[s["op"]](s)


def _map(s):
    if own:
        positions, slots = s["plan"].token_map()
        return {"positions": positions, "slots": slots}
    t = torch.arange(s["T"], device="cuda")
    i = torch.searchsorted(s["qo"][1:], t, right=True)
    P = s["L"][i] - s["n"][i] + t - s["qo"][i]
    return {"positions": P, "slots": s["table"][i, P // s["page"]] * s["page"] + P % s["page"]}


def _rotate(s, x):
    """x [T, heads, D] with the pairs of its first R dims turned by their angles, in 32 bits."""
    R = s["rotary"]
    angle = s["positions"].double()[:, None, None] * s["freq"]
    c, n = torch.cos(angle).float(), torch.sin(angle).float()
    y = x.float()
    a, b = (y[..., 0:R:2], y[..., 1:R:2]) if s["interleaved"] else (y[..., :R // 2], y[..., R // 2:R])
    a, b = a * c - b * n, b * c + a * n
    turned = torch.stack((a, b), -1).flatten(-2) if s["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((turned, y[..., R:]), -1)


def _rope(s):
    if own:
        import paged_kv_attention_slot_gb300 as pk
        q = pk.rope_store(s["q"], s["kn"], s["vn"], s["positions"], s["slots"], s["cache"], s["rotary_of"])
        return {"q": q, **_as_values(s)}
    page, off = s["slots"] // s["page"], s["slots"] % s["page"]
    k, v = _rotate(s, s["kn"]), s["vn"].float()
    if s["dtype"] == "e4m3":
        k = (k * (1.0 / s["k_scale"])).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v * (1.0 / s["v_scale"])).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s["k"][page, off], s["v"][page, off] = k.to(s["k"].dtype), v.to(s["v"].dtype)
    return {"q": _rotate(s, s["q"]).to(torch.bfloat16), **_as_values(s)}


def _as_values(s):
    return {n: s[n] if s["dtype"] == "bf16" else s[n].view(torch.float8_e4m3fn) for n in ("k", "v")}


def _wide(s, n, x, sf):
    """The values of pool rows of K (or V) in 32 bits."""
    if s["dtype"] == "bf16":
        return x.float()
    scale = torch.tensor(s[n + "_scale"], dtype=torch.float32, device="cuda")
    if s["dtype"] == "e4m3":
        return x.view(torch.float8_e4m3fn).float() * scale
    table = torch.tensor(E2M1 + tuple(-e for e in E2M1), dtype=torch.float32, device="cuda")
    c = torch.stack((x & 15, x >> 4), -1).flatten(-2)
    return (table[c.int()].unflatten(-1, (-1, 16)) * sf.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2) * scale


def _bound(s):
    if own:
        s["plan"].bound_keys(s["cache"], s["bounds"], all_pages=s.get("every", False))
        return {"codes": s["codes"]}
    page = s["page"]
    N = (s["L"] + page - 1) // page
    if s.get("every", False):
        at = torch.arange(len(s["pages"]), device="cuda")
        i = torch.searchsorted(s["indptr"][1:], at, right=True)
        block = at - s["indptr"][i]
    else:
        i, block = torch.arange(len(N), device="cuda"), N - 1
    pages = s["table"][i, block]
    x = _wide(s, "k", s["k"][pages], s["k_sf"][pages] if s["dtype"] == "nvfp4" else None)  # [pages, page, H, D]
    there = (block[:, None] * page + torch.arange(page, device="cuda") < s["L"][i][:, None])[:, :, None, None]
    lo = torch.floor(x.masked_fill(~there, math.inf).amin(1) / s["scale"])
    hi = torch.ceil(x.masked_fill(~there, -math.inf).amax(1) / s["scale"])
    s["codes"][pages] = torch.stack((lo, hi), 2).clamp(-127, 127).to(torch.int8)
    return {"codes": s["codes"]}


def _best(s, score):
    """The blocks that are attended to, ascending, -1 behind them: [B, H, blocks] from score [B, H, most]."""
    K, S, R, most = s["blocks"], s["sink"], s["recent"], s["most"]
    N = ((s["L"] + s["page"] - 1) // s["page"])[:, None, None]
    b = torch.arange(most, device="cuda").expand(score.shape)
    body = (b >= S) & (b < N - R)
    order = torch.sort(score.double().masked_fill(~body, -math.inf), dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, b)
    keep = (b < N) & ((N <= K) | (b < S) | (b >= N - R) | (body & (rank < K - S - R)))
    first = torch.sort(torch.where(keep, b, most), dim=-1).values
    first = torch.cat((first, torch.full((*score.shape[:2], max(0, K - most)), most, device="cuda")), -1)[..., :K]
    return torch.where(first < most, first, -1).int()


def _select(s):
    if own:
        return {"blocks": s["plan"].select(s["q"], s["bounds"], num_sink=s["sink"], num_recent=s["recent"])}
    H, G = s["kv_heads"], s["heads"] // s["kv_heads"]
    # whole-number weights: codes of the queries in units of the largest of the group's
    a = s["q"].float().unflatten(1, (H, G)) * s["scale"][:, None, :]
    m = a.abs().amax((2, 3), keepdim=True)
    c = torch.round(a / torch.where(m > 0, m, 1.0) * float(32767 // G)).double()
    w = torch.cat((c.clamp(max=0).sum(2), c.clamp(min=0).sum(2)), -1)  # [B, H, 2 D]: for the lower, for the upper bound
    codes = s["codes"][s["table"]].double().flatten(-2).transpose(1, 2)  # [B, H, most, 2 D]
    return {"blocks": _best(s, torch.matmul(codes, w.unsqueeze(-1)).squeeze(-1))}


def _attend(s):
    if own:
        o, lse = s["plan"].run(s["q"], s["cache"], return_lse=True, blocks=s["chosen"])
        return {"o": o, "lse": lse}
    B, Hq, D = s["q"].shape
    H, page = s["kv_heads"], s["page"]
    chosen = s["chosen"].long()
    there = (chosen * page)[..., None] + torch.arange(page, device="cuda") < s["L"][:, None, None, None]
    there = (there & (chosen >= 0)[..., None]).flatten(-2)  # [B, H, keys]
    rows = torch.gather(s["table"][:, None].expand(B, H, -1), 2, chosen.clamp(min=0))
    head = torch.arange(H, device="cuda")[None, :, None]
    k, v = (_wide(s, n, s[n][rows, :, head], s[n + "_sf"][rows, :, head] if s["dtype"] == "nvfp4" else None).flatten(2, 3)
            for n in ("k", "v"))
    x = torch.matmul(s["q"].float().view(B, H, Hq // H, D), k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    x = x.masked_fill(~there[:, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    return {"o": torch.matmul(p / l, v).reshape(B, Hq, D).to(torch.bfloat16), "lse": (m + torch.log(l)).reshape(B, Hq)}


def _step(s):
    codes = _bound(s)["codes"]
    s["chosen"] = _select(s)["blocks"]
    return {"codes": codes, "blocks": s["chosen"], **_attend(s)}


# ------------------------------------------------------------------------------------------------
# from the definition, in 64 bits
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "map":
        L, n = _lengths(case)
        table = s["table"].cpu().numpy()
        at = [(i, p) for i in range(len(L)) for p in range(int(L[i] - n[i]), int(L[i]))]
        slots = [int(table[i, p // case["page"]]) * case["page"] + p % case["page"] for i, p in at]
        return {"positions": torch.tensor([p for _, p in at], dtype=torch.int64), "slots": torch.tensor(slots, dtype=torch.int64)}
    if case["op"] == "rope":
        return _exact_rope(case, s)
    if case["op"] == "bound":
        return {"codes": _exact_codes(case, s)}
    if case["op"] == "select":
        return {"blocks": _exact_blocks(case, s)}
    if case["op"] == "attend":
        return _exact_attend(case, s, s["chosen"])
    s["codes"] = _exact_codes(case, s)
    chosen = _exact_blocks(case, s)
    return {"codes": s["codes"], "blocks": chosen, **_exact_attend(case, s, chosen)}


def _exact_rope(case, s):
    freq = torch.from_numpy(_frequencies(case)).cuda()
    unit = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double().outer(freq))[:, None]
    half = case["rotary"] // 2

    def turn(x):
        y = x.double().clone()
        r = y[..., :case["rotary"]]
        pairs = r.unflatten(-1, (half, 2)) if case["interleaved"] else r.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
        y[..., :case["rotary"]] = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return y

    r = {"q": turn(s["q"])}
    at = (s["slots"] // case["page"], s["slots"] % case["page"])
    for n, x in (("k", turn(s["kn"])), ("v", s["vn"].double())):
        r[n] = torch.zeros(s[n].shape, dtype=torch.float64, device="cuda")
        r[n][at] = x if case["dtype"] == "bf16" else (x / s[n + "_scale"]).clamp(-448, 448)
    return r


def _exact_rows(s, n, page, at, head):
    """Values of the keys (values) at the offsets `at` of one page and head, in 64 bits."""
    x = s[n][page, at, head]
    if s["dtype"] == "bf16":
        return x.double()
    scale = float(np.float32(s[n + "_scale"]))
    if s["dtype"] == "e4m3":
        return x.view(torch.float8_e4m3fn).double() * scale
    c = torch.stack((x % 16, x // 16), -1).flatten(-2).double()
    m, e, sign = c % 2, torch.floor(c / 2) % 4, 1 - 2 * torch.floor(c / 8)
    f = s[n + "_sf"][page, at, head].view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    return torch.where(e == 0, 0.5 * m, torch.exp2(e - 1) * (1 + 0.5 * m)) * sign * f * scale


def _exact_codes(case, s):
    out, page = s["codes"].clone(), case["page"]
    for i, n in enumerate(s["L"].tolist()):
        blocks = -(-n // page)
        for full in (True, False):  # the whole pages together, the last one by itself
            if full and not case.get("every", False):
                continue
            ids = s["table"][i, :blocks - 1] if full else s["table"][i, blocks - 1:blocks]
            if not len(ids):
                continue
            off = torch.arange(page if full else n - (blocks - 1) * page, device="cuda")
            x = _exact_rows(s, "k", ids[:, None], off[None, :], slice(None))  # [pages, keys, H, D]
            # (the quotient is defined in float32, whole numbers from there)
            lo, hi = torch.floor(x.amin(1).float() / s["scale"]), torch.ceil(x.amax(1).float() / s["scale"])
            out[ids] = torch.stack((lo, hi), 2).clamp(-127, 127).to(torch.int8)
    return out


def _exact_blocks(case, s):
    H, K, S, R, page = case["kv_heads"], case["blocks"], case["sink"], case["recent"], case["page"]
    G = case["heads"] // H
    q, scale = s["q"].float().cpu().numpy(), s["scale"].cpu().numpy()
    codes, table = s["codes"].cpu().numpy(), s["table"].cpu().numpy()
    out = np.full((len(q), H, K), -1, dtype=np.int32)
    for i, n in enumerate(s["L"].tolist()):
        N = -(-n // page)
        if N <= K:
            out[i, :, :N] = np.arange(N)
            continue
        for h in range(H):
            # (products and quotients are defined in float32, whole numbers from there)
            a = q[i, h * G:(h + 1) * G] * scale[h]
            c = np.rint(a / np.abs(a).max() * np.float32(32767 // G)).astype(np.int64)
            bound = codes[table[i, S:N - R], h].astype(np.int64)
            score = bound[:, 0] @ np.minimum(c, 0).sum(0) + bound[:, 1] @ np.maximum(c, 0).sum(0)
            best = np.lexsort((np.arange(len(score)), -score))[:K - S - R] + S
            out[i, h] = np.concatenate([np.arange(S), np.sort(best), np.arange(N - R, N)])
    return torch.from_numpy(out)


def _exact_attend(case, s, chosen):
    H, page, D = case["kv_heads"], case["page"], case["dim"]
    G = case["heads"] // H
    o = torch.empty((len(s["q"]), case["heads"], D), dtype=torch.float64, device="cuda")
    lse = torch.empty(o.shape[:2], dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["L"].tolist()):
        for h in range(H):
            b = chosen[i, h].to("cuda").long()
            b = b[b >= 0]
            pos = (b[:, None] * page + torch.arange(page, device="cuda")).flatten()
            pos = pos[pos < n]
            ids, off = s["table"][i, pos // page], pos % page
            x = s["q"][i, h * G:(h + 1) * G].double() @ _exact_rows(s, "k", ids, off, h).t() / math.sqrt(D)
            lse[i, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            o[i, h * G:(h + 1) * G] = torch.softmax(x, -1) @ _exact_rows(s, "v", ids, off, h)
    return {"o": o, "lse": lse}
