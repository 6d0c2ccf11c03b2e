"""What the operators around a compressed cache cost, and what they compute.

Three operators that a serving or training program calls next to the cache's own path:

* rotary positions on queries, tokens and attention outputs (``csa_rotary``);
* copying, forking, compacting and freeing the blocks of cache slots (``csa_cache_copy``);
* dense attention of many queries over one compressed prefix that they share, joined with
  each query's own part (``hca_shared_attend``).

``run`` computes them with elementary torch operations where ``own`` is false and calls
``fp4_kv_cache_csa_b200`` where it is true. ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
KEY_FORMATS = ("none", "bf16", "e4m3", "mxfp4")


def listed():
    return [
        # one decode step: the queries of 32 requests at up to 1M tokens, the last 64 of 512 channels rotated
        dict(name="rotary_decode", op="rotary", rows=32, heads=64, dim=512, rot=64, half=False, inverse=False,
             x="bf16", out="bf16", far=1 << 20, scaled=1.0),
        # the queries of a prefill chunk
        dict(name="rotary_prefill", op="rotary", rows=8192, heads=64, dim=512, rot=64, half=False, inverse=False,
             x="bf16", out="bf16", far=1 << 17, scaled=4.0),
        # attention outputs turned back (entries are both key and value) and rounded for the next product
        dict(name="rotary_back_f32", op="rotary", rows=4001, heads=16, dim=512, rot=64, half=True, inverse=True,
             x="f32", out="bf16", far=1 << 20, scaled=1.0),
        # the gradient of rotated tokens of a training batch: whole vectors, half layout, 32 bits
        dict(name="rotary_gradient", op="rotary", rows=30011, heads=4, dim=128, rot=128, half=True, inverse=True,
             x="f32", out="f32", far=1 << 15, scaled=8.0),
        # one finished 1M-token prompt (HCA, 8192 blocks) forked to 32 continuations
        dict(name="fork_hca", op="copy", jobs=32, blocks=8192, cap=8256, dim=512, e4m3=False, key="none", idx=0,
             keep=0, fan=32),
        # two 1M-token CSA requests moved to two slots each of another cache
        dict(name="fork_csa_1m", op="copy", jobs=4, blocks=262143, cap=262144, dim=512, e4m3=False, key="e4m3",
             idx=128, keep=0, fan=2),
        # a cache cut down to the 512 blocks that an indexer kept of each of eight 64K-token requests
        dict(name="compact_topk", op="copy", jobs=8, blocks=16384, cap=16384, dim=512, e4m3=True, key="mxfp4",
             idx=128, keep=512, fan=1),
        # half of every block list of 32 long requests evicted
        dict(name="compact_half", op="copy", jobs=32, blocks=131072, cap=131072, dim=512, e4m3=False, key="bf16",
             idx=64, keep=65521, fan=1),
        # four samples of a short prompt in a small model
        dict(name="shared_tiny", op="attend", groups=1, queries=4, blocks=1024, dim=128, heads=16, e4m3=False,
             causal=0, join=True, ragged=False),
        # 32 samples of one 1M-token prompt decoding over its 8192 HCA blocks
        dict(name="shared_decode", op="attend", groups=1, queries=32, blocks=8192, dim=512, heads=64, e4m3=False,
             causal=0, join=True, ragged=False),
        # samples of four prompts of different lengths, the other scale format
        dict(name="shared_ragged", op="attend", groups=4, queries=61, blocks=7001, dim=512, heads=64, e4m3=True,
             causal=0, join=True, ragged=True),
        # a causal prefill chunk attended densely over 64K tokens compressed 4x
        dict(name="shared_causal", op="attend", groups=1, queries=512, blocks=16384, dim=512, heads=64, e4m3=False,
             causal=4, join=False, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "copy", "attend"))
    if op == "rotary":
        dim = rng.choice((64, 128, 512))
        rot = rng.choice([r for r in (32, 64, 128) if r <= dim])
        heads = rng.choice((1, 3, 4, 16, 64))
        rows = min(_log(rng, 1, 8192), (1 << 28) // (heads * dim))
        return dict(op=op, rows=rows, heads=heads, dim=dim, rot=rot, half=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, x=rng.choice(("bf16", "f32")), out=rng.choice(("bf16", "f32")),
                    far=_log(rng, 1 << 12, 1 << 20), scaled=rng.choice((1.0, 4.0, 40.0)))
    if op == "copy":
        jobs = _log(rng, 1, 32)
        blocks = _log(rng, 1, min(262144, 2097152 // jobs))
        key = rng.choice(KEY_FORMATS)
        return dict(op=op, jobs=jobs, blocks=blocks, cap=blocks + rng.randrange(0, 70), dim=rng.choice((128, 512)),
                    e4m3=rng.random() < 0.5, key=key, idx=0 if key == "none" else rng.choice((64, 128)),
                    keep=rng.choice((0, rng.randint(1, blocks))), fan=rng.randint(1, jobs))
    dim = rng.choice((128, 512, 512))
    heads = rng.choice((16, 64, 64, 40))
    groups = rng.randint(1, 4)
    blocks = _log(rng, 1, 16384)
    queries = max(groups, min(_log(rng, 1, 512), (512 * 16384 * 64 // 2) // (blocks * heads * groups)))
    return dict(op=op, groups=groups, queries=queries, blocks=blocks, dim=dim, heads=heads, e4m3=rng.random() < 0.5,
                causal=rng.choice((0, 0, 4, 128)), join=rng.random() < 0.5, ragged=rng.random() < 0.5)


# ---------------------------------------------------------------- sizes that a case fixes
def _copy_lengths(c):
    """Blocks of each of the slots that are copied from: a few of them shorter."""
    n = -(-c["jobs"] // c["fan"])
    return [max(1, c["blocks"] - (37 * i) % 64) for i in range(n)]


def _copy_counts(c):
    """Blocks that each job keeps."""
    lens = _copy_lengths(c)
    return [min(c["keep"] or c["blocks"], lens[j // c["fan"]]) for j in range(c["jobs"])]


def _attend_sizes(c):
    """Queries of each prefix, and its blocks."""
    g, q = c["groups"], c["queries"]
    if not c["ragged"]:
        return [q // g + (i < q % g) for i in range(g)], [c["blocks"]] * g
    w = [2 * i + 1 for i in range(g)]
    counts = [q * x // sum(w) for x in w]
    counts[-1] += q - sum(counts)
    return counts, [max(1, c["blocks"] * (g - i) // g - 13 * i) for i in range(g)]


def _attend_visible(c):
    """For each prefix the blocks that its queries see: the newest query sees all of them."""
    counts, blocks = _attend_sizes(c)
    m = c["causal"]
    if not m:
        return [[n] * k for k, n in zip(counts, blocks)]
    return [[max(0, n * m - (k - 1 - i)) // m for i in range(k)] for k, n in zip(counts, blocks)]


def _row_bytes(c):
    key = {"none": 0, "bf16": 2 * c["idx"], "e4m3": c["idx"], "mxfp4": c["idx"] // 2 + c["idx"] // 32}[c["key"]]
    return c["dim"] // 2 + c["dim"] // (16 if c["e4m3"] else 32) + key


def work(case):
    c = case
    if c["op"] == "rotary":
        n = c["rows"] * c["heads"] * c["dim"]
        size = {"bf16": 2, "f32": 4}
        return {"bytes": n * (size[c["x"]] + size[c["out"]]) + 4 * c["rows"],
                "flops": 3 * c["rows"] * c["heads"] * c["rot"]}
    if c["op"] == "copy":
        counts = _copy_counts(c)
        if c["keep"]:
            read = sum(counts) * (_row_bytes(c) + 4)  # every job its own list of blocks
        else:
            read = sum(_copy_lengths(c)) * _row_bytes(c)  # each source slot once, however often it is forked
        return {"bytes": read + sum(counts) * _row_bytes(c), "flops": 0}
    counts, blocks = _attend_sizes(c)
    row = c["dim"] // 2 + c["dim"] // (16 if c["e4m3"] else 32)
    vec = c["queries"] * c["heads"]
    size = 2 * vec * c["dim"] * 2 + 4 * vec + (4 * vec * (c["dim"] + 1) if c["join"] else 0)
    seen = sum(sum(v) for v in _attend_visible(c))
    return {"bytes": sum(blocks) * row + size, "flops": 4 * seen * c["heads"] * c["dim"]}


# ---------------------------------------------------------------- inputs
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _planes(c, g, slots):
    """Cache planes with the bytes that pooled tokens leave: any codes, scales of a few binades."""
    dev, cap = "cuda", c["cap"]

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device=dev, dtype=torch.uint8)

    p = {"fp4": ints(0, 256, slots, cap, c["dim"] // 2)}
    p["scale"] = (ints(0x1C, 0x2C, slots, cap, c["dim"] // 16) if c["e4m3"]
                  else ints(123, 127, slots, cap, c["dim"] // 32))
    key, idx = c.get("key", "none"), c.get("idx", 0)
    p["idx_key"] = p["idx_key_scale"] = None
    if key == "bf16":
        p["idx_key"] = torch.randn(slots, cap, idx, generator=g, device=dev, dtype=torch.bfloat16)
    elif key == "e4m3":
        p["idx_key"] = ints(0, 0x7F, slots, cap, idx)
    elif key == "mxfp4":
        p["idx_key"] = ints(0, 256, slots, cap, idx // 2)
        p["idx_key_scale"] = ints(122, 127, slots, cap, idx // 32)
    return p


def _cache(p, n_blocks, block):
    import fp4_kv_cache_csa_b200 as csa

    kind = csa.CSA_IDX_BF16
    if p["idx_key_scale"] is not None:
        kind = csa.CSA_IDX_MXFP4
    elif p["idx_key"] is not None and p["idx_key"].dtype == torch.uint8:
        kind = csa.CSA_IDX_E4M3
    fmt = csa.CSA_SCALE_E4M3_16 if p["e4m3"] else csa.CSA_SCALE_E8M0_32
    return csa.Cache(fp4=p["fp4"], scale=p["scale"], n_blocks=n_blocks, block=block, idx_key=p["idx_key"],
                     idx_dtype=kind, scale_fmt=fmt, idx_key_scale=p["idx_key_scale"])


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    if c["op"] == "rotary":
        x = torch.randn(c["rows"], c["heads"], c["dim"], generator=g, device=dev).to(_dtype(c["x"]))
        pos = torch.randint(0, c["far"], (c["rows"],), generator=g, device=dev, dtype=torch.int32)
        p = torch.arange(c["rot"] // 2, dtype=torch.float64)
        inv = (10000.0 ** (-2.0 * p / c["rot"]) / c["scaled"]).to(torch.float32).to(dev)
        return {"case": c, "x": x, "pos": pos, "inv": inv, "mscale": 1.0 + 0.1 * math.log(c["scaled"])}
    if c["op"] == "copy":
        lens = _copy_lengths(c)
        src = _planes(c, g, len(lens))
        src["e4m3"] = c["e4m3"]
        dst = {k: torch.zeros(c["jobs"], *v.shape[1:], dtype=v.dtype, device=dev) if torch.is_tensor(v) else v
               for k, v in src.items()}
        src_slot = torch.arange(c["jobs"], device=dev, dtype=torch.int32) // c["fan"]
        dst_slot = torch.randperm(c["jobs"], generator=g, device=dev).to(torch.int32)
        keep = None
        if c["keep"]:  # ascending, -1 behind the last one, as the indexer's selections are
            keep = torch.full((c["jobs"], c["keep"]), -1, dtype=torch.int32, device=dev)
            for j, n in enumerate(_copy_counts(c)):
                pick = torch.randperm(lens[j // c["fan"]], generator=g, device=dev)[:n]
                keep[j, :n] = pick.sort().values.to(torch.int32)
        return {"case": c, "src": src, "dst": dst, "src_n": torch.tensor(lens, dtype=torch.int32, device=dev),
                "dst_n": torch.zeros(c["jobs"], dtype=torch.int32, device=dev), "src_slot": src_slot,
                "dst_slot": dst_slot, "keep": keep}
    counts, blocks = _attend_sizes(c)
    d = dict(c, cap=max(blocks))
    p = _planes(d, g, c["groups"])
    p["e4m3"] = c["e4m3"]
    q = torch.randn(c["queries"], c["heads"], c["dim"], generator=g, device=dev).to(torch.bfloat16)
    offs = [0]
    for k in counts:
        offs.append(offs[-1] + k)
    s = {"case": c, "planes": p, "q": q, "counts": counts, "blocks": blocks,
         "n_blocks": torch.tensor(blocks, dtype=torch.int32, device=dev),
         "q_offsets": torch.tensor(offs, dtype=torch.int32, device=dev), "q_pos": None, "join_out": None,
         "join_lse": None}
    if c["causal"]:
        m = c["causal"]
        pos = [n * m - 1 - (k - 1 - i) for k, n in zip(counts, blocks) for i in range(k)]
        s["q_pos"] = torch.tensor(pos, dtype=torch.int32, device=dev).clamp_(min=0)
    if c["join"]:  # what attention over a query's own newest tokens returned
        s["join_out"] = 0.3 * torch.randn(q.shape, generator=g, device=dev)
        s["join_lse"] = 5.0 + torch.randn(q.shape[:2], generator=g, device=dev)
    return s


# ---------------------------------------------------------------- one pass
def _run_rotary(s):
    c, x = s["case"], s["x"]
    if own:
        import fp4_kv_cache_csa_b200 as csa

        return csa.csa_rotary(x, s["pos"], s["inv"], layout=csa.CSA_ROPE_HALF if c["half"] else csa.CSA_ROPE_PAIRS,
                              inverse=c["inverse"], mscale=s["mscale"], out_dtype=_dtype(c["out"]))
    lead, y = x[..., : c["dim"] - c["rot"]], x[..., c["dim"] - c["rot"]:].float()
    angle = s["pos"].double()[:, None, None] * s["inv"].double()
    cos, sin = (torch.cos(angle) * s["mscale"]).float(), (torch.sin(angle) * s["mscale"]).float()
    if c["inverse"]:
        sin = -sin
    if c["half"]:
        a, b = y[..., : c["rot"] // 2], y[..., c["rot"] // 2:]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    else:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    return torch.cat((lead.to(_dtype(c["out"])), y.to(_dtype(c["out"]))), -1)


PLANES = ("fp4", "scale", "idx_key", "idx_key_scale")


def _run_copy(s):
    src, dst = s["src"], s["dst"]
    if own:
        import fp4_kv_cache_csa_b200 as csa

        csa.csa_cache_copy(_cache(src, s["src_n"], 4), _cache(dst, s["dst_n"], 4), s["src_slot"], s["dst_slot"],
                           keep=s["keep"])
    else:
        a, b = s["src_slot"].long(), s["dst_slot"].long()
        if s["keep"] is None:
            n = s["src_n"][a]
            live = torch.arange(src["fp4"].shape[1], device=n.device)[None, :, None] < n[:, None, None]
        else:
            live = (s["keep"] >= 0)[..., None]
            n = live[..., 0].sum(1, dtype=torch.int32)
        for name in PLANES:
            if src[name] is not None:
                k = live.shape[1]
                rows = src[name][a] if s["keep"] is None else src[name][a[:, None], s["keep"].clamp(min=0).long()]
                dst[name][b, :k] = torch.where(live, rows, dst[name][b, :k])
        s["dst_n"][b] = n
    # the stored bits themselves: a copy has to keep every one of them
    planes = [dst[name] for name in PLANES if dst[name] is not None]
    return [x.view(torch.int16) if x.dtype == torch.bfloat16 else x for x in planes] + [s["dst_n"]]


def _entries(p, b, n, dtype):
    """The first n blocks of slot b as numbers."""
    codes = p["fp4"][b, :n]
    lut = torch.tensor(E2M1, device=codes.device, dtype=dtype)
    e = torch.stack((lut[(codes & 15).long()], lut[(codes >> 4).long()]), -1).flatten(-2)
    raw = p["scale"][b, :n]
    sc = raw.view(torch.float8_e4m3fn).to(dtype) if p["e4m3"] else torch.exp2(raw.to(dtype) - 127)
    return (e.view(n, raw.shape[1], -1) * sc[..., None]).flatten(1)


def _run_attend(s):
    c, q, p = s["case"], s["q"], s["planes"]
    scale = c["dim"] ** -0.5
    if own:
        import fp4_kv_cache_csa_b200 as csa

        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        out = csa.hca_shared_attend(_cache(p, s["n_blocks"], c["causal"] or 128), q, s["q_offsets"], s["q_pos"],
                                    join_out=s["join_out"], join_lse=s["join_lse"], softmax_scale=scale, lse=lse)
        return out, lse
    outs, lses, at = [], [], 0
    for b, (k, n) in enumerate(zip(s["counts"], s["blocks"])):  # one prefix after the other
        if not k:
            continue
        e = _entries(p, b, n, torch.float32)
        u = (q[at: at + k].float().flatten(0, 1) @ e.T).view(k, -1, n) * scale
        if c["causal"]:
            seen = ((s["q_pos"][at: at + k] + 1) // c["causal"])[:, None, None]
            u = u.masked_fill(torch.arange(n, device=u.device) >= seen, -math.inf)
        top = u.amax(-1, keepdim=True).clamp(min=-1e30)
        w = torch.exp(u - top)
        total = w.sum(-1, keepdim=True)
        lse = (torch.log(total) + top)[..., 0]
        o = (w.flatten(0, 1) @ e).view(k, -1, c["dim"]) / total.clamp(min=1e-30)
        if c["join"]:
            other = s["join_lse"][at: at + k]
            both = torch.logaddexp(lse, other)
            o = (o * torch.exp(lse - both)[..., None]
                 + s["join_out"][at: at + k] * torch.exp(other - both)[..., None])
            lse = both
        outs.append(o.to(torch.bfloat16))
        lses.append(lse)
        at += k
    return torch.cat(outs), torch.cat(lses)


def run(state):
    return {"rotary": _run_rotary, "copy": _run_copy, "attend": _run_attend}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_rotary(s):
    c = s["case"]
    x = s["x"].double()
    first, r = c["dim"] - c["rot"], c["rot"] // 2
    out = x.clone()
    unit = torch.polar(torch.full((c["rows"], r), s["mscale"], dtype=torch.float64, device=x.device),
                       (-1.0 if c["inverse"] else 1.0) * torch.outer(s["pos"].double(), s["inv"].double()))
    ia = first + (torch.arange(r) if c["half"] else 2 * torch.arange(r))
    ib = ia + (r if c["half"] else 1)
    z = torch.complex(x[:, :, ia], x[:, :, ib]) * unit[:, None, :]
    out[:, :, ia], out[:, :, ib] = z.real, z.imag
    return out


def _exact_attend(s):
    c, counts, blocks = s["case"], s["counts"], s["blocks"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    i = 0
    for b, seen in enumerate(_attend_visible(c)):
        if not seen:
            continue
        e = _entries(s["planes"], b, blocks[b], torch.float64)
        for j in range(0, len(seen), 8):  # eight queries at a time
            n = seen[j: j + 8]
            q = s["q"][i + j: i + j + len(n)].double()
            u = torch.matmul(q, e.T) / math.sqrt(c["dim"])
            hidden = torch.arange(blocks[b], device="cuda")[None] >= torch.tensor(n, device="cuda")[:, None]
            u.masked_fill_(hidden[:, None, :], -math.inf)
            total = torch.logsumexp(u, -1)
            w = torch.nan_to_num(torch.exp(u - total[..., None]))
            lse[i + j: i + j + len(n)] = total
            out[i + j: i + j + len(n)] = torch.matmul(w, e)
        i += len(seen)
    if c["join"]:
        other = s["join_lse"].double()
        share = torch.sigmoid(lse - other)[..., None]
        out = share * out + (1 - share) * s["join_out"].double()
        lse = torch.logaddexp(lse, other)
    return out, lse


def exact(case, seed):
    if case["op"] == "copy":
        return None  # bytes and counts only
    s = prepare(case, seed)
    return _exact_rotary(s) if case["op"] == "rotary" else _exact_attend(s)
