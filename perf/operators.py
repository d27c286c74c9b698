"""What is measured of the paged-cache operators: the cases, their inputs, their plain forms and their definition.

Four operators share one paged key/value cache (pages [num_pages][Hkv][page][D], a page table per sequence):

  append   q, k, v of T tokens (rows of one fused projection) are rotated by their positions, on one axis or on three
           (time, height, width), and k, v are stored to the cache
  decode   one query token per sequence against its pages
  prefix   the same for a batch whose sequences all begin with one shared prefix
  prefill  the new tokens of each sequence, causally, against the cache that holds them already

``run`` computes them in elementary torch operations, or, with ``own`` set, through the package's entry points.
"""

import math

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one token of one sequence in a decode loop: the fp32 rows of the fused projection (launch latency)
        dict(name="append_1_token", op="append", src="f32", dtype="f16", B=1, H=32, Hkv=8, D=128, page=16, new_lo=1,
             new_hi=1, ctx_lo=511, ctx_hi=511, axes=1, rot=128, layout="half", base=10000.0),
        # a decode batch, odd in number, far positions, half of each head rotated in neighbouring pairs
        dict(name="append_57_tokens_far", op="append", src="bf16", dtype="bf16", B=57, H=32, Hkv=4, D=128, page=64,
             new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=999, axes=1, rot=64, layout="pairs", base=1000000.0,
             pos0=100000),
        # prompts with images among the text: three axes, two ragged prompts
        dict(name="append_prompt_3_axes", op="append", src="f32", dtype="bf16", B=2, H=32, Hkv=8, D=128, page=32,
             new_lo=3001, new_hi=4096, ctx_lo=0, ctx_hi=77, axes=3, rot=128, layout="half", base=1000000.0),
        # a page of text, 12 heads of 64 (latency)
        dict(name="decode_page_12_heads", op="decode", dtype="f16", B=1, H=12, Hkv=12, D=64, page=16, len_lo=512,
             len_hi=512, out16=False),
        # a 7B-shaped decode batch, grouped heads, lengths all over the range, some sequences already ended
        dict(name="decode_7b_gqa_ragged", op="decode", dtype="f16", B=48, H=32, Hkv=8, D=128, page=16, len_lo=0,
             len_hi=8191, out16=True),
        # one long sequence
        dict(name="decode_one_long", op="decode", dtype="bf16", B=1, H=32, Hkv=8, D=128, page=64, len_lo=100003,
             len_hi=100003, out16=False),
        # multi-head, the most bytes
        dict(name="decode_7b_mha", op="decode", dtype="f16", B=16, H=32, Hkv=32, D=128, page=32, len_lo=4096,
             len_hi=4096, out16=False),
        # a few requests behind one system prompt
        dict(name="prefix_small", op="prefix", dtype="f16", B=7, H=32, Hkv=8, D=128, page=16, prefix=1021, len_lo=1,
             len_hi=64, out16=False),
        # a full batch behind a long document
        dict(name="prefix_large", op="prefix", dtype="bf16", B=128, H=32, Hkv=8, D=128, page=64, prefix=16384,
             len_lo=1, len_hi=500, out16=True),
        # drafted tokens of a few sequences checked against their caches
        dict(name="prefill_drafts", op="prefill", dtype="f16", B=4, H=32, Hkv=8, D=128, page=16, new_lo=3, new_hi=6,
             ctx_lo=900, ctx_hi=2100, out16=False),
        # ragged prompts, heads of 64, one part of them cached before
        dict(name="prefill_ragged_64", op="prefill", dtype="f16", B=5, H=12, Hkv=12, D=64, page=16, new_lo=1,
             new_hi=1500, ctx_lo=0, ctx_hi=700, out16=False),
        # one long prompt, 7B-shaped, grouped heads
        dict(name="prefill_8192", op="prefill", dtype="bf16", B=1, H=32, Hkv=8, D=128, page=64, new_lo=8192,
             new_hi=8192, ctx_lo=0, ctx_hi=0, out16=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefix", "prefill"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8, 8, 12])
    G = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 16])
    case = dict(op=op, dtype=rng.choice(["f16", "bf16"]), H=Hkv * G, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]))
    if op == "append":
        B = _log_int(rng, 1, 64)
        new = 1 if rng.random() < 0.4 else _log_int(rng, 1, max(1, 200000 // (B * Hkv * (G + 2))))
        ctx = _log_int(rng, 1, 2000)
        case.update(src=rng.choice(["f32", "f16", "bf16"]), B=B, new_lo=max(1, new // 2), new_hi=new, ctx_lo=ctx // 3,
                    ctx_hi=ctx, axes=rng.choice([1, 1, 3]), rot=rng.choice([D, D, D // 2]),
                    layout=rng.choice(["half", "pairs"]), base=rng.choice([10000.0, 500000.0]),
                    pos0=rng.choice([0, 0, 1000000]))
        return case
    case["out16"] = rng.random() < 0.5
    if op == "prefill":
        B = _log_int(rng, 1, 12)
        new = _log_int(rng, 2, max(2, min(3000, 100000 // (Hkv * G)) // B))
        ctx = _log_int(rng, 1, 3000)
        case.update(B=B, new_lo=max(1, new // 3), new_hi=new, ctx_lo=0, ctx_hi=ctx)
        return case
    B = _log_int(rng, 1, 96)
    hi = _log_int(rng, 1, max(64, min(40000, 1200000 // (B * Hkv))))
    case.update(B=B, len_lo=rng.choice([0, 1, hi]), len_hi=hi)
    case["len_lo"] = min(case["len_lo"], hi)
    if op == "prefix":
        case.update(prefix=_log_int(rng, 16, 20000), len_hi=min(hi, 700), len_lo=min(case["len_lo"], hi, 700))
    return case


def _spread(n, lo, hi, salt):
    """n whole numbers of [lo, hi], scattered, the last of them hi: the sizes belong to the case, not to the seed."""
    out = [lo + ((i + 1) * 2654435761 + salt * 40503 >> 7) % (hi - lo + 1) for i in range(n)]
    out[-1] = hi
    return out


def _sizes(case):
    """(new tokens, private tokens in the cache) of each sequence."""
    B = case["B"]
    if case["op"] in ("append", "prefill"):
        new = _spread(B, case["new_lo"], case["new_hi"], 1)
        ctx = _spread(B, case["ctx_lo"], case["ctx_hi"], 2)
        return new, [a + b for a, b in zip(new, ctx)]
    return [1] * B, _spread(B, case["len_lo"], case["len_hi"], 3)


def _sections(case):
    half = case["rot"] // 2
    return [half] if case["axes"] == 1 else [half // 4, half - half // 4 - half // 3, half // 3]


_arena = []


def _reserve(lwq, nbytes, dev):
    """One workspace for every state, registered once and again when a state needs more."""
    if not _arena or _arena[-1].numel() < nbytes:
        _arena.append(torch.empty(max(nbytes, 64 << 20), dtype=torch.uint8, device=dev))
        lwq.lwq_init(_arena[-1], _arena[-1].numel())


def _inputs(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7919 + 17)
    t = _TYPES[case["dtype"]]
    B, H, Hkv, D, page = (case[k] for k in ("B", "H", "Hkv", "D", "page"))
    new, lens = _sizes(case)
    T, P = sum(new), case.get("prefix", 0)
    max_pages = max(1, max(-(-n // page) for n in lens))
    npre = -(-P // page)
    count = sum(-(-n // page) for n in lens) + npre + 3
    perm = torch.randperm(count, generator=g, device=dev).to(torch.int32)
    s = dict(case, new=new, lens=lens, T=T, P=P, max_pages=max_pages, num_pages=count)
    tables = torch.zeros((B, max_pages), dtype=torch.int32, device=dev)
    at = npre
    for b, n in enumerate(lens):
        k = -(-n // page)
        tables[b, :k] = perm[at:at + k]
        at += k
    s["tables"], s["prefix_pages"] = tables, perm[:npre].contiguous()
    s["lens_d"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"], s["cu_d"] = cu, torch.tensor(cu, dtype=torch.int32, device=dev)
    s["kc"] = torch.randn((count, Hkv, page, D), generator=g, device=dev, dtype=t)
    s["vc"] = torch.randn((count, Hkv, page, D), generator=g, device=dev, dtype=t)
    if case["op"] == "append":
        s["qkv"] = torch.randn((T, (H + 2 * Hkv) * D), generator=g, device=dev, dtype=_TYPES[case["src"]])
        s["q_out"] = torch.zeros((T, H, D), dtype=t, device=dev)
        own_pos = torch.cat([torch.arange(n - m, n, device=dev) for m, n in zip(new, lens)]).to(torch.int32)
        pos = own_pos.repeat(case["axes"], 1) + case.get("pos0", 0)
        if case["axes"] == 3:  # an image's patches: rows and columns beside the time
            pos[1] += torch.randint(0, 64, (T,), generator=g, device=dev, dtype=torch.int32)
            pos[2] += torch.randint(0, 64, (T,), generator=g, device=dev, dtype=torch.int32)
        s["pos"] = pos.contiguous()
    else:
        s["q"] = torch.randn((T, H, D), generator=g, device=dev, dtype=t)
        s["out"] = torch.zeros((T, H, D), dtype=t if case["out16"] else torch.float32, device=dev)
        s["scale"] = D ** -0.5
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import block_quantized_matmul_lwq_b200 as lwq
        act = lwq.ACT_DTYPES[case["dtype"]]
        s["cache"] = lwq.lwq_paged(act, s["kc"], s["vc"], s["tables"], s["lens_d"], B=case["B"], Hkv=case["Hkv"],
                                   D=case["D"], page=case["page"], max_pages=s["max_pages"],
                                   num_pages=s["num_pages"], prefix=s["prefix_pages"] if s["P"] else None,
                                   prefix_len=s["P"])
        if case["op"] == "append":
            s["rope"] = lwq.lwq_rope_init(case["rot"], base=case["base"], sections=_sections(case),
                                          layout=lwq.LWQ_ROPE_HALF if case["layout"] == "half" else lwq.LWQ_ROPE_PAIRS)
        elif case["op"] == "prefill":
            _reserve(lwq, lwq.lwq_attention_prefill_workspace_size(s["cache"], s["T"], case["H"]), s["q"].device)
        else:
            _reserve(lwq, lwq.lwq_attention_paged_workspace_size(s["cache"], case["H"]), s["q"].device)
    return s


def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    import block_quantized_matmul_lwq_b200 as lwq
    stream = torch.cuda.current_stream()
    H, Hkv, D = s["H"], s["Hkv"], s["D"]
    if s["op"] == "append":
        x, ld = s["qkv"], (H + 2 * Hkv) * D
        lwq.lwq_kv_append(s["cache"], s["rope"], lwq.ACT_DTYPES[s["src"]], x, ld, x[:, H * D:], ld,
                          x[:, (H + Hkv) * D:], ld, s["q_out"], s["T"], H, cu_tokens=s["cu_d"], positions=s["pos"],
                          stream=stream)
        return [s["q_out"], s["kc"], s["vc"]]
    flags = lwq.LWQ_FLAG_OUT16 if s["out16"] else 0
    if s["op"] == "prefill":
        lwq.lwq_attention_prefill(s["cache"], s["q"], s["out"], s["cu_d"], s["T"], H, s["scale"], flags=flags,
                                  stream=stream)
    else:
        lwq.lwq_attention_paged(s["cache"], s["q"], s["out"], H, s["scale"], flags=flags, stream=stream)
    return s["out"]


# ---------------------------------------------------------------- plain forms
def _slots(s):
    """Page and offset of every new token, in the tokens' order."""
    page = s["page"]
    pages, offs = [], []
    for b, (m, n) in enumerate(zip(s["new"], s["lens"])):
        j = torch.arange(n - m, n, device=s["tables"].device)
        pages.append(s["tables"][b][j // page])
        offs.append(j % page)
    return torch.cat(pages).long(), torch.cat(offs)


def _rotate(x, cos, sin, rot, layout):
    """x [T][heads][D] in 32 bits; cos, sin [T][1][rot / 2]."""
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_append(s):
    T, H, Hkv, D, rot = s["T"], s["H"], s["Hkv"], s["D"], s["rot"]
    x = s["qkv"].float().view(T, H + 2 * Hkv, D)
    i = torch.arange(rot // 2, device=x.device, dtype=torch.float64)
    freq = s["base"] ** (-2.0 * i / rot)
    axis = torch.cat([torch.full((n,), a, device=x.device) for a, n in enumerate(_sections(s))])
    ang = s["pos"].double()[axis].t() * freq          # [T][rot / 2], in 64 bits: far positions
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    s["q_out"].copy_(_rotate(x[:, :H], cos, sin, rot, s["layout"]))
    k = _rotate(x[:, H:H + Hkv], cos, sin, rot, s["layout"])
    page, off = _slots(s)
    s["kc"][page, :, off] = k.to(s["kc"].dtype)
    s["vc"][page, :, off] = x[:, H + Hkv:].to(s["vc"].dtype)
    return [s["q_out"], s["kc"], s["vc"]]


def _gather(cache, pages, n):
    """The first n tokens of a page list in 32 bits: [Hkv][n][D]."""
    x = cache[pages.long()]                            # [pages][Hkv][page][D]
    x = x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])
    return x[:, :n].float()


def _softmax_weights(scores, keep=None):
    if keep is not None:
        scores = scores.masked_fill(~keep, float("-inf"))
    top = scores.amax(-1, keepdim=True).clamp_min(-1e30)
    w = (scores - top).exp()
    return w, w.sum(-1, keepdim=True)


def _plain_decode(s):
    B, H, Hkv, D, page = s["B"], s["H"], s["Hkv"], s["D"], s["page"]
    G = H // Hkv
    q = s["q"].float().view(B, Hkv, G, D) * s["scale"]
    rows = []
    if s["P"]:  # the prefix once for the batch: its scores, and its weighted values by each row's own top
        pk, pv = _gather(s["kc"], s["prefix_pages"], s["P"]), _gather(s["vc"], s["prefix_pages"], s["P"])
        ps = torch.matmul(q.permute(1, 0, 2, 3).reshape(Hkv, B * G, D), pk.transpose(1, 2)).view(Hkv, B, G, -1)
    for b, n in enumerate(s["lens"]):
        if n + s["P"] == 0:
            rows.append(torch.zeros((Hkv, G, D), device=q.device))
            continue
        k, v = _gather(s["kc"], s["tables"][b], n), _gather(s["vc"], s["tables"][b], n)
        sc = torch.matmul(q[b], k.transpose(1, 2))
        if s["P"]:
            w, total = _softmax_weights(torch.cat([ps[:, b], sc], -1))
            acc = torch.matmul(w[..., :s["P"]], pv) + torch.matmul(w[..., s["P"]:], v)
        else:
            w, total = _softmax_weights(sc)
            acc = torch.matmul(w, v)
        rows.append(acc / total)
    s["out"].copy_(torch.stack(rows).view(B, H, D))
    return s["out"]


def _plain_prefill(s):
    H, Hkv, D = s["H"], s["Hkv"], s["D"]
    G = H // Hkv
    for b, (m, n) in enumerate(zip(s["new"], s["lens"])):
        t0 = s["cu"][b]
        k, v = _gather(s["kc"], s["tables"][b], n), _gather(s["vc"], s["tables"][b], n)
        q = s["q"][t0:t0 + m].float() * s["scale"]
        seen = torch.arange(n, device=q.device)[None] <= torch.arange(n - m, n, device=q.device)[:, None]
        for h in range(Hkv):
            sc = torch.matmul(q[:, h * G:(h + 1) * G].transpose(0, 1), k[h].t())   # [G][m][n]
            w, total = _softmax_weights(sc, seen)
            s["out"][t0:t0 + m, h * G:(h + 1) * G] = (torch.matmul(w, v[h]) / total).transpose(0, 1).to(s["out"].dtype)
    return s["out"]


_PLAIN = {"append": _plain_append, "decode": _plain_decode, "prefix": _plain_decode, "prefill": _plain_prefill}


# ----------------------------------------------------------------- definition
def exact(case, seed):
    """The outputs in 64 bits from the definition, token by token of the cache's flat slots."""
    s = _inputs(case, seed)
    H, Hkv, D, page = s["H"], s["Hkv"], s["D"], s["page"]
    G = H // Hkv
    dev = s["tables"].device

    def flat(b, n):  # slots of the first n private tokens of sequence b
        j = torch.arange(n, device=dev)
        return s["tables"][b].long()[torch.div(j, page, rounding_mode="floor")] * page + torch.remainder(j, page)

    if case["op"] == "append":
        rot, T = s["rot"], s["T"]
        x = s["qkv"].double().view(T, H + 2 * Hkv, D)
        freq = torch.exp(torch.arange(0, rot, 2, device=dev, dtype=torch.float64) * (-math.log(s["base"]) / rot))
        which = [a for a, n in enumerate(_sections(case)) for _ in range(n)]
        ang = torch.stack([s["pos"][a].double() * freq[i] for i, a in enumerate(which)], 1)
        turn = torch.polar(torch.ones_like(ang), ang)[:, None]
        qk = x[:, :H + Hkv].clone()
        if s["layout"] == "half":
            z = torch.complex(qk[..., :rot // 2], qk[..., rot // 2:rot]) * turn
            qk[..., :rot // 2], qk[..., rot // 2:rot] = z.real, z.imag
        else:
            z = torch.view_as_complex(qk[..., :rot].reshape(T, H + Hkv, rot // 2, 2).contiguous()) * turn
            qk[..., :rot] = torch.view_as_real(z).reshape(T, H + Hkv, rot)
        kc, vc = s["kc"].double(), s["vc"].double()
        slot = torch.cat([flat(b, n)[n - m:] for b, (m, n) in enumerate(zip(s["new"], s["lens"]))])
        kc.permute(0, 2, 1, 3)[slot // page, slot % page] = qk[:, H:]
        vc.permute(0, 2, 1, 3)[slot // page, slot % page] = x[:, H + Hkv:]
        return [qk[:, :H].contiguous(), kc, vc]

    pages = torch.arange(s["P"], device=dev)
    pre = s["prefix_pages"].long()[pages // page] * page + pages % page if s["P"] else pages
    out = torch.zeros((s["T"], H, D), dtype=torch.float64, device=dev)
    for b, (m, n) in enumerate(zip(s["new"], s["lens"])):
        slot = torch.cat([pre, flat(b, n)])
        if slot.numel() == 0:
            continue
        P = s["P"]
        visible = torch.arange(slot.numel(), device=dev)[None] < (P + n - m + 1 + torch.arange(m, device=dev))[:, None]
        if case["op"] != "prefill":
            visible = torch.ones_like(visible)
        rows = slice(s["cu"][b], s["cu"][b + 1])
        for h in range(Hkv):
            k = s["kc"][slot // page, h, slot % page].double()
            v = s["vc"][slot // page, h, slot % page].double()
            for g in range(h * G, (h + 1) * G):
                sc = (s["q"][rows, g].double() @ k.t()) * s["scale"]
                sc = torch.where(visible, sc, torch.full_like(sc, -math.inf))
                w = torch.exp(sc - torch.logsumexp(sc, 1, keepdim=True))
                out[rows, g] = w @ v
    return out


def work(case):
    new, lens = _sizes(case)
    H, Hkv, D, T, B = case["H"], case["Hkv"], case["D"], sum(new), case["B"]
    if case["op"] == "append":
        src = 4 if case["src"] == "f32" else 2
        data = T * (H + 2 * Hkv) * D * (src + 2)
        index = 4 * (T * case["axes"] + 2 * B + 1 + sum(-(-n // case["page"]) for n in lens))
        return {"bytes": data + index, "flops": 3 * T * (H + Hkv) * case["rot"]}
    P = case.get("prefix", 0)
    kv = (P + sum(lens)) * Hkv * D * 2 * 2
    index = 4 * (B + (P + sum(lens)) // case["page"])
    io = T * H * D * (2 + (2 if case["out16"] else 4))
    if case["op"] == "prefill":
        pairs = sum(m * (n - m) + m * (m + 1) // 2 for m, n in zip(new, lens))
    else:
        pairs = B * P + sum(lens)
    return {"bytes": kv + io + index, "flops": 4 * H * D * pairs}
