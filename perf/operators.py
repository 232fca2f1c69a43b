"""Performance cases of the query/key preparation and of attention over key blocks chosen for each query.

The operators, in the order in which a layer or a decoding step calls them:

  rope      qk_norm_rope           per-head RMS norm of Q and K, position rotation, head-major rows (into a cache)
  ropegrad  qk_norm_rope_backward  its gradient
  mean      block_mean             the mean key of every block of keys (all blocks, or those the newest tokens touch)
  select    block_select           for every query the `topk` blocks with the largest q . mean
  attn      block_attn             softmax attention of every query over the keys of its blocks
  attngrad  block_attn_backward    its gradient

Shapes: G = Hq / Hk query heads share a key head and its blocks; Nq new tokens end a context of kv_len keys, kept in
buffers of Nk rows; token n of a sequence has position kv_len - Nq + n.
"""
import math

import torch

own = False      # set by the measuring tools: run() makes the framework's calls

EPS = 1e-6
CHUNK = 1 << 28          # fp32 values that the plain attention gathers at a time


# ------------------------------------------------------------------------------------------------ cases
def _case(name, op, **kw):
    c = dict(name=name, op=op, B=1, Hq=8, Hk=8, D=128, Nq=1, Nk=1, block=64, topk=16, sink=1, local=2, causal=True,
             ragged=False, interleaved=False, new=0)
    c.update(kw)
    return c


def listed():
    return [
        # one decoding step of 16 sequences: the new tokens' rows go to each sequence's place in the cache
        _case("rope_decode", "rope", B=16, Hq=40, Hk=8, Nq=1, Nk=2000, ragged=True),
        # the 480p, 5 s layer: 21x30x52 tokens, 40 heads, rotation of neighbouring pairs
        _case("rope_480p", "rope", Hq=40, Hk=40, Nq=32760, Nk=32760, interleaved=True),
        # a fine-tuning step, shared key heads, an odd length
        _case("rope_grad", "ropegrad", B=2, Hq=32, Hk=8, D=64, Nq=5001, Nk=5001),
        # block means of a whole 480p, 5 s layer (ragged last block)
        _case("mean_480p", "mean", Hq=40, Hk=40, Nq=32760, Nk=32760),
        # block means after one decoding step of 16 sequences
        _case("mean_append", "mean", B=16, Hq=40, Hk=8, Nq=1, Nk=16384, ragged=True, new=1),
        # block choice for every token of a 32,760-token prompt or clip
        _case("select_prefill", "select", Hq=40, Hk=8, Nq=32760, Nk=32760),
        # block choice of one decoding step over long caches
        _case("select_decode", "select", B=16, Hq=40, Hk=8, Nk=131072, topk=32, ragged=True),
        # attention of one decoding step over long caches
        _case("attn_decode", "attn", B=16, Hq=40, Hk=8, Nk=32768, topk=32, ragged=True),
        # a video layer (8 of its heads), every query sees all frames
        _case("attn_480p", "attn", Hq=8, Hk=8, Nq=32760, Nk=32760, topk=32, causal=False),
        # left-padded causal prompts, shared key heads
        _case("attn_causal", "attn", B=2, Hq=40, Hk=8, Nq=8190, Nk=8190, ragged=True),
        # gradient of a causal layer with shared key heads
        _case("grad_causal", "attngrad", Hq=40, Hk=8, Nq=8190, Nk=8190),
        # gradient of a small layer, own key heads, 128-key blocks, ragged batch, D = 64
        _case("grad_ragged", "attngrad", B=3, Hq=12, Hk=12, D=64, Nq=1999, Nk=1999, block=128, topk=6, causal=False,
              ragged=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "ropegrad", "mean", "select", "attn", "attngrad"])
    D = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    B = rng.choice([1, 2, 3, 8, 16])
    block = rng.choice([64, 128])
    topk = _spread(rng, 4, 32)
    decode = rng.random() < 0.4
    ragged = rng.random() < 0.5
    kw = dict(B=B, Hq=Hk * G, Hk=Hk, D=D, block=block, topk=topk, sink=rng.choice([0, 1, 2]), local=rng.choice([1, 2]),
              causal=rng.random() < 0.6, ragged=ragged, interleaved=rng.random() < 0.5)
    rows = B * Hk                                   # key heads of the batch
    if op in ("rope", "ropegrad"):
        heads = B * Hk * (G + 2)
        most = min(32760, 32760 * 120 // heads if op == "rope" else 5001 * 80 // heads)
        n = rng.randint(1, 4) if decode else _spread(rng, min(16, most), most)
        return _case("", op, **{**kw, "Nq": n, "Nk": n + (rng.randint(0, 999) if op == "rope" else 0)})
    if op == "mean":
        nk = _spread(rng, 100, min(32760, 32760 * 40 // rows))
        return _case("", op, **{**kw, "Nq": 1, "Nk": nk, "new": rng.randint(1, 5) if decode else 0})
    if decode and op != "attngrad":
        nk = _spread(rng, 1000, min(131072, 32768 * 128 // rows))
        return _case("", op, **{**kw, "Nq": rng.randint(1, 4), "Nk": nk, "causal": True})
    # work of all queries: rows * n^2 / block scores, rows * G * n * topk * block attended keys
    most = 32760.0
    if op == "select":
        most = min(most, math.sqrt(8 * 32760.0 ** 2 / rows))
    else:
        keys = 8 * 32760.0 * 32 * 64 if op == "attn" else 8190.0 * 40 * 16 * 64
        most = min(most, keys / (rows * G * topk * block), (8190 if op == "attngrad" else 32760) * 8.0 / rows)
    n = _spread(rng, min(100, most), most)
    return _case("", op, **{**kw, "Nq": n, "Nk": n})


def _lens(c):
    """Context length of every sequence of the batch."""
    if not c["ragged"]:
        return [c["Nk"]] * c["B"]
    least = c["Nq"] if c["op"] == "rope" else 1
    return [max(least, c["Nk"] - b * (c["Nk"] // (2 * c["B"])) - b % 7) for b in range(c["B"])]


def _blocks(c):
    return -(-c["Nk"] // c["block"])


# ------------------------------------------------------------------------------------------------ inputs
def _tokens(c, g, lens):
    """Q [B*Hq, Nq, D], K and V [B*Hk, Nk, D]: passages (or tiles of a clip) of 192 tokens, each about one of a few
    topics; Q and K of a token are its topic's centre plus noise.  Rows behind a sequence hold what was there before."""
    dev = dict(device="cuda", generator=g)
    B, Hq, Hk, D, Nq, Nk = c["B"], c["Hq"], c["Hk"], c["D"], c["Nq"], c["Nk"]
    topics = max(4, Nk // 1024)
    seg = torch.randint(topics, (B * Hk, Nk // 192 + 1), **dev)
    label = seg[:, torch.arange(Nk, device="cuda") // 192]
    centre = torch.randn(B * Hk, topics, D, **dev)
    head = torch.arange(B * Hk, device="cuda")[:, None]
    k = centre[head, label].add_(torch.randn(B * Hk, Nk, D, **dev), alpha=0.5).bfloat16()
    v = torch.randn(B * Hk, Nk, D, **dev).bfloat16()
    pos = torch.tensor(lens, device="cuda").repeat_interleave(Hk)[:, None] - Nq + torch.arange(Nq, device="cuda")
    mine = centre[head, label.gather(1, pos.clamp_min(0))]
    q = mine[:, None] + torch.randn(B * Hk, Hq // Hk, Nq, D, **dev) * 0.5
    return q.bfloat16().view(B * Hq, Nq, D), k, v


def _means(c, k, lens):
    n, nb = c["block"], _blocks(c)
    t = torch.tensor(lens, device="cuda").repeat_interleave(c["Hk"])[:, None]
    x = k.float() * (torch.arange(c["Nk"], device="cuda") < t)[..., None]
    x = torch.nn.functional.pad(x, (0, 0, 0, nb * n - c["Nk"])).view(k.shape[0], nb, n, c["D"]).sum(2)
    count = (t - torch.arange(nb, device="cuda") * n).clamp(0, n)
    return x / count.clamp_min(1)[..., None]


def _choose(c, scores, lens):
    """Block lists [B*Hk, Nq, topk] of scores [B*Hk, Nq, blocks]: ascending, filled up with -1."""
    dev = scores.device
    t = torch.tensor(lens, device=dev).repeat_interleave(c["Hk"])[:, None]
    pos = t - c["Nq"] + torch.arange(c["Nq"], device=dev)
    seen = pos + 1 if c["causal"] else t.expand_as(pos)
    j = torch.arange(scores.shape[2], device=dev)
    mine = torch.div(pos, c["block"], rounding_mode="floor")[..., None]
    may = j * c["block"] < seen[..., None]
    must = may & ((j < c["sink"]) | ((j <= mine) & (j > mine - c["local"])))
    key = torch.where(must, math.inf, torch.where(may, scores, -math.inf))
    key, at = torch.sort(key, dim=2, descending=True, stable=True)
    at = torch.where(key > -math.inf, at, 1 << 30)
    at = at[..., : c["topk"]].sort(2).values
    at = torch.nn.functional.pad(at, (0, c["topk"] - at.shape[2]), value=1 << 30)
    return torch.where(at < 1 << 30, at, -1).int()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, Hq, Hk, D, Nq, Nk = c["B"], c["Hq"], c["Hk"], c["D"], c["Nq"], c["Nk"]
    lens = _lens(c)
    s = {"case": c, "lens": lens, "kv_len": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    rnd = lambda *shape: torch.randn(*shape, device="cuda", generator=g)  # noqa: E731
    if c["op"] in ("rope", "ropegrad"):
        # one projection's output: the heads of Q, K and V of a token side by side
        qkv = (rnd(B, Nq, Hq + 2 * Hk, D) * 1.5).bfloat16()
        s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:]
        s["w_q"], s["w_k"] = 1 + 0.2 * rnd(D), 1 + 0.2 * rnd(D)
        angle = torch.arange(Nk, device="cuda").double()[:, None] * 10000.0 ** (
            -torch.arange(D // 2, device="cuda").double() / (D // 2))
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["start"] = s["kv_len"] - Nq if c["op"] == "rope" and Nk > Nq else None
        s["q_out"] = torch.empty(B * Hq, Nq, D, dtype=torch.bfloat16, device="cuda")
        if c["op"] == "rope":
            s["k_out"], s["v_out"] = rnd(B * Hk, Nk, D).bfloat16(), rnd(B * Hk, Nk, D).bfloat16()
        else:
            s["dq_out"] = rnd(B * Hq, Nq, D).bfloat16()
            s["dk_out"], s["dv_out"] = rnd(B * Hk, Nk, D).bfloat16(), rnd(B * Hk, Nk, D).bfloat16()
        return s
    s["q"], s["k"], s["v"] = _tokens(c, g, lens)
    mean = _means(c, s["k"], lens)
    if c["op"] == "mean":
        s["mean"] = mean
        if c["new"]:         # the means before the newest tokens came
            s["mean"] = _means(c, s["k"], [max(0, n - c["new"]) for n in lens])
        s.pop("q"), s.pop("v")
        return s
    if c["op"] == "select":
        s["mean"] = mean
        s.pop("k"), s.pop("v")
        s["sel"] = torch.empty(B * Hk, Nq, c["topk"], dtype=torch.int32, device="cuda")
        return s
    qs = s["q"].float().view(B * Hk, Hq // Hk, Nq, D).sum(1)
    s["sel"] = _choose(c, qs @ mean.transpose(1, 2), lens)
    if c["op"] == "attngrad":
        o, lse = _attend(s)
        s["o"], s["lse"] = o, lse
        s["do"] = rnd(B * Hq, Nq, D).bfloat16()
    return s


# ------------------------------------------------------------------------------------------------ the plain forms
def _rotate(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _positions(s):
    c = s["case"]
    first = torch.zeros(c["B"], dtype=torch.int32, device="cuda") if s["start"] is None else s["start"]
    return (first[:, None] + torch.arange(c["Nq"], device="cuda")).long()        # [B, Nq]


def _rope(s):
    c = s["case"]
    pos = _positions(s)
    cos, sin = s["cos"][pos][:, :, None], s["sin"][pos][:, :, None]

    def head_rows(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        return _rotate(x, cos, sin, c["interleaved"]).bfloat16().transpose(1, 2)         # [B, H, Nq, D]

    s["q_out"].view(c["B"], c["Hq"], c["Nq"], c["D"]).copy_(head_rows(s["q"], s["w_q"]))
    at = pos[:, None, :, None].expand(c["B"], c["Hk"], c["Nq"], c["D"])
    cache = (c["B"], c["Hk"], c["Nk"], c["D"])
    s["k_out"].view(cache).scatter_(2, at, head_rows(s["k"], s["w_k"]))
    s["v_out"].view(cache).scatter_(2, at, s["v"].transpose(1, 2))
    return s["q_out"], s["k_out"], s["v_out"]


def _rope_grad(s):
    c = s["case"]
    pos = _positions(s)
    cos, sin = s["cos"][pos][:, :, None], s["sin"][pos][:, :, None]

    def back(x, w, d, H):
        x = x.float()
        g = _rotate(d.view(c["B"], H, c["Nq"], c["D"]).transpose(1, 2).float(), cos, -sin, c["interleaved"])
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        n = x * r
        dw = (g * n).sum((0, 1, 2), dtype=torch.float64).float()
        g = g * w
        return (r * (g - n * (g * n).mean(-1, keepdim=True))).bfloat16(), dw

    dq, dw_q = back(s["q"], s["w_q"], s["dq_out"], c["Hq"])
    dk, dw_k = back(s["k"], s["w_k"], s["dk_out"], c["Hk"])
    dv = s["dv_out"].view(c["B"], c["Hk"], c["Nk"], c["D"]).transpose(1, 2).contiguous()
    return dq, dk, dv, dw_q, dw_k


def _mean(s):
    c = s["case"]
    if not c["new"]:
        return _means(c, s["k"], s["lens"])
    t = s["kv_len"].long().repeat_interleave(c["Hk"])[:, None]
    blk = (t - c["new"]).clamp_min(0) // c["block"] + torch.arange((c["new"] + c["block"] - 2) // c["block"] + 1,
                                                                   device="cuda")
    row = blk[..., None] * c["block"] + torch.arange(c["block"], device="cuda")
    head = torch.arange(row.shape[0], device="cuda")
    x = s["k"][head[:, None, None], row.clamp_max(c["Nk"] - 1)].float() * (row < t[..., None])[..., None]
    x = x.sum(2) / (t - blk * c["block"]).clamp(1, c["block"])[..., None]
    last = blk.clamp_max(_blocks(c) - 1)
    old = s["mean"][head[:, None], last]
    x = torch.where((blk * c["block"] < t)[..., None], x, old)
    s["mean"][head[:, None], last] = torch.where((blk == last)[..., None], x, s["mean"][head[:, None], last])
    return s["mean"]


def _select(s):
    # scores next to the border decide between blocks: 64 bits
    c = s["case"]
    qs = s["q"].double().view(-1, c["Hq"] // c["Hk"], c["Nq"], c["D"]).sum(1)
    return _choose(c, qs @ s["mean"].double().transpose(1, 2), s["lens"])


def _chosen_keys(s, h, n):
    """Key rows [rows, topk * block] of the queries n of key heads h, and which of them the query sees."""
    c = s["case"]
    t = s["kv_len"].long()[h // c["Hk"]]
    seen = t - c["Nq"] + n + 1 if c["causal"] else t
    sel = s["sel"][h, n].long()
    key = sel[..., None] * c["block"] + torch.arange(c["block"], device="cuda")
    ok = (sel[..., None] >= 0) & (key < seen[:, None, None])
    return key.flatten(1).clamp(0, c["Nk"] - 1), ok.flatten(1)


def _row_chunks(c):
    per = max(1, CHUNK // (c["topk"] * c["block"] * c["D"]))
    return torch.arange(c["B"] * c["Hk"] * c["Nq"], device="cuda").split(per)


def _attend(s):
    c = s["case"]
    G, Nq, D = c["Hq"] // c["Hk"], c["Nq"], c["D"]
    q = s["q"].view(-1, G, Nq, D)

    def rows(r):
        h, n = r // Nq, r % Nq
        key, ok = _chosen_keys(s, h, n)
        a = (q[h, :, n].float() @ s["k"][h[:, None], key].float().transpose(1, 2)) / math.sqrt(D)
        a = torch.where(ok[:, None], a, -math.inf)
        top = a.amax(-1, keepdim=True)
        top = torch.where(top > -math.inf, top, 0.0)
        p = torch.exp(a - top)
        total = p.sum(-1, keepdim=True)
        o = (p @ s["v"][h[:, None], key].float()) / torch.where(total > 0, total, 1.0)
        return o.bfloat16(), (top + torch.log(total))[..., 0]

    o, lse = (torch.cat(x) for x in zip(*[rows(r) for r in _row_chunks(c)]))
    return (o.view(-1, Nq, G, D).transpose(1, 2).reshape(-1, Nq, D),
            lse.view(-1, Nq, G).transpose(1, 2).reshape(-1, Nq))


def _attend_grad(s):
    c = s["case"]
    G, Nq, Nk, D = c["Hq"] // c["Hk"], c["Nq"], c["Nk"], c["D"]
    q, do, o = (s[x].view(-1, G, Nq, D) for x in ("q", "do", "o"))
    lse = s["lse"].view(-1, G, Nq)
    dk = torch.zeros(c["B"] * c["Hk"] * Nk, D, device="cuda")
    dv = torch.zeros_like(dk)

    def rows(r):
        h, n = r // Nq, r % Nq
        key, ok = _chosen_keys(s, h, n)
        qr, dr = q[h, :, n].float(), do[h, :, n].float()
        kk = s["k"][h[:, None], key].float()
        a = (qr @ kk.transpose(1, 2)) / math.sqrt(D)
        p = torch.where(ok[:, None], torch.exp(a - lse[h, :, n][..., None]), 0.0)
        dp = dr @ s["v"][h[:, None], key].float().transpose(1, 2)
        ds = p * (dp - (dr * o[h, :, n].float()).sum(-1, keepdim=True)) / math.sqrt(D)
        at = (h[:, None] * Nk + key).flatten()
        dk.index_add_(0, at, (ds.transpose(1, 2) @ qr).view(-1, D))
        dv.index_add_(0, at, (p.transpose(1, 2) @ dr).view(-1, D))
        return (ds @ kk).bfloat16()

    dq = torch.cat([rows(r) for r in _row_chunks(c)])
    return (dq.view(-1, Nq, G, D).transpose(1, 2).reshape(-1, Nq, D), dk.bfloat16().view(-1, Nk, D),
            dv.bfloat16().view(-1, Nk, D))


_PLAIN = {"rope": _rope, "ropegrad": _rope_grad, "mean": _mean, "select": _select, "attn": _attend,
          "attngrad": _attend_grad}


def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------ the framework's calls
def _svg():
    import sparse_attention_long_svg_b200 as svg
    return svg


def _own_rope(s):
    return _svg().qk_norm_rope(s["q"], s["k"], s["v"], s["w_q"], s["w_k"], s["cos"], s["sin"], eps=EPS,
                               interleaved=s["case"]["interleaved"], start=s["start"], q_out=s["q_out"],
                               k_out=s["k_out"], v_out=s["v_out"])


def _own_rope_grad(s):
    return _svg().qk_norm_rope_backward(s["dq_out"], s["dk_out"], s["dv_out"], s["q"], s["k"], s["w_q"], s["w_k"],
                                        s["cos"], s["sin"], eps=EPS, interleaved=s["case"]["interleaved"],
                                        start=s["start"])


def _own_mean(s):
    c = s["case"]
    return _svg().block_mean(s["k"], c["block"], kv_len=s["kv_len"], new=c["new"], mean=s["mean"] if c["new"] else None)


def _own_select(s):
    c = s["case"]
    return _svg().block_select(s["q"], s["mean"], c["block"], c["topk"], c["Nk"], sink=c["sink"], local=c["local"],
                               causal=c["causal"], kv_len=s["kv_len"], sel=s["sel"])


def _own_attn(s):
    c = s["case"]
    return _svg().block_attn(s["q"], s["k"], s["v"], s["sel"], c["block"], causal=c["causal"], kv_len=s["kv_len"],
                             want_lse=True)


def _own_attn_grad(s):
    c = s["case"]
    return _svg().block_attn_backward(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["sel"], c["block"],
                                      causal=c["causal"], kv_len=s["kv_len"])


_OWN = {"rope": _own_rope, "ropegrad": _own_rope_grad, "mean": _own_mean, "select": _own_select, "attn": _own_attn,
        "attngrad": _own_attn_grad}


# ------------------------------------------------------------------------------------------------ work
def _pairs(c):
    """(query, visible key) pairs of one query head, and key rows that one key head's queries read at least once."""
    pairs = rows = 0
    for n in _lens(c):
        for i in range(c["Nq"]):
            seen = min(n, n - c["Nq"] + i + 1) if c["causal"] else n
            if seen <= 0:
                continue
            whole, rest = divmod(seen, c["block"])
            if whole + (rest > 0) <= c["topk"]:
                pairs += seen
            elif rest and c["local"] and (c["causal"] or i + 1 == c["Nq"]):
                pairs += (c["topk"] - 1) * c["block"] + rest
            else:
                pairs += c["topk"] * c["block"]
        rows += min(n, c["Nq"] * c["topk"] * c["block"])
    return pairs, rows


def work(case):
    c = case
    B, Hq, Hk, D, Nq, Nk = c["B"], c["Hq"], c["Hk"], c["D"], c["Nq"], c["Nk"]
    nb = _blocks(c)
    if c["op"] in ("rope", "ropegrad"):
        tokens = B * Nq
        table = min(tokens, Nk) * D * 4
        if c["op"] == "rope":
            return {"bytes": tokens * (Hq + 2 * Hk) * D * 2 * 2 + table + 8 * D, "flops": tokens * (Hq + Hk) * D * 8}
        return {"bytes": tokens * (3 * (Hq + Hk) + 2 * Hk) * D * 2 + table + 16 * D,
                "flops": tokens * (Hq + Hk) * D * 16}
    if c["op"] == "mean":
        if c["new"]:
            first = [max(0, n - c["new"]) // c["block"] * c["block"] for n in _lens(c)]
            rows = sum(n - f for n, f in zip(_lens(c), first))
            out = sum(-(-n // c["block"]) - f // c["block"] for n, f in zip(_lens(c), first))
        else:
            rows, out = sum(_lens(c)), B * nb
        return {"bytes": Hk * (rows * D * 2 + out * D * 4), "flops": Hk * rows * D}
    if c["op"] == "select":
        scores = 0
        for n in _lens(c):
            if c["causal"]:
                scores += sum(max(0, (n - Nq + i) // c["block"] + 1) for i in range(Nq))
            else:
                scores += Nq * -(-n // c["block"])
        means = sum(-(-n // c["block"]) for n in _lens(c))
        return {"bytes": B * Hq * Nq * D * 2 + Hk * means * D * 4 + B * Hk * Nq * c["topk"] * 4,
                "flops": Hk * scores * 2 * D}
    pairs, rows = _pairs(c)
    lists = B * Hk * Nq * c["topk"] * 4
    q_rows = B * Hq * Nq * D * 2
    if c["op"] == "attn":
        return {"bytes": 2 * q_rows + Hk * rows * D * 2 * 2 + lists + B * Hq * Nq * 4, "flops": Hq * pairs * 4 * D}
    return {"bytes": 4 * q_rows + Hk * rows * D * 2 * 2 + B * Hk * Nk * D * 2 * 2 + lists + B * Hq * Nq * 4,
            "flops": Hq * pairs * 10 * D}


# ------------------------------------------------------------------------------------------------ in 64 bits, from the definitions
def _turn(x, pos, s, back=False):
    """Rotation as a product of complex numbers."""
    c = s["case"]
    z = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, :, None]         # [B, Nq, 1, D/2]
    z = z.conj() if back else z
    x = x.unflatten(-1, (-1, 2)) if c["interleaved"] else x.unflatten(-1, (2, -1)).transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(x.contiguous()) * z)
    return y.flatten(-2) if c["interleaved"] else y.transpose(-1, -2).flatten(-2)


def _exact_rope(s):
    c = s["case"]
    first = [0] * c["B"] if s["start"] is None else [n - c["Nq"] for n in s["lens"]]
    pos = torch.tensor(first, device="cuda")[:, None] + torch.arange(c["Nq"], device="cuda")
    norm = lambda x: x.double() / (x.double().pow(2).sum(-1, keepdim=True) / c["D"] + EPS).sqrt()  # noqa: E731
    q = _turn(norm(s["q"]) * s["w_q"].double(), pos, s).permute(0, 2, 1, 3).reshape(-1, c["Nq"], c["D"])
    k = _turn(norm(s["k"]) * s["w_k"].double(), pos, s)
    k_out, v_out = s["k_out"].double(), s["v_out"].double()
    for b, p in enumerate(first):
        heads = slice(b * c["Hk"], (b + 1) * c["Hk"])
        k_out[heads, p:p + c["Nq"]] = k[b].transpose(0, 1)
        v_out[heads, p:p + c["Nq"]] = s["v"][b].transpose(0, 1).double()
    return q, k_out, v_out


def _exact_rope_grad(s):
    c = s["case"]
    pos = torch.arange(c["Nq"], device="cuda").expand(c["B"], -1)

    def back(x, w, d, H):
        x, w = x.double(), w.double()
        u = _turn(d.double().view(c["B"], H, c["Nq"], c["D"]).permute(0, 2, 1, 3), pos, s, back=True)
        var = x.pow(2).sum(-1, keepdim=True) / c["D"] + EPS
        # y = w x var^-1/2:  dx = w u var^-1/2 - x (sum w u x) var^-3/2 / D
        dx = w * u * var ** -0.5 - x * (w * u * x).sum(-1, keepdim=True) * var ** -1.5 / c["D"]
        return dx, torch.einsum("bnhd,bnhd->d", u, x * var ** -0.5)

    dq, dw_q = back(s["q"], s["w_q"], s["dq_out"], c["Hq"])
    dk, dw_k = back(s["k"], s["w_k"], s["dk_out"], c["Hk"])
    return dq, dk, s["dv_out"].double().view(c["B"], c["Hk"], c["Nq"], c["D"]).permute(0, 2, 1, 3), dw_q, dw_k


def _exact_mean(s):
    c = s["case"]
    out = s["mean"].double() if c["new"] else torch.zeros_like(s["mean"], dtype=torch.float64)
    for b, n in enumerate(s["lens"]):
        heads = slice(b * c["Hk"], (b + 1) * c["Hk"])
        k = s["k"][heads, :n].double()
        first = max(0, n - c["new"]) // c["block"] if c["new"] else 0
        for j in range(first, -(-n // c["block"])):
            out[heads, j] = k[:, j * c["block"]:(j + 1) * c["block"]].mean(1)
    return out


def _exact_select(s):
    """A block is kept when fewer blocks beat it than there are places."""
    c = s["case"]
    G, nb = c["Hq"] // c["Hk"], _blocks(c)
    j = torch.arange(nb, device="cuda")
    out = torch.full(s["sel"].shape, -1, dtype=torch.int32, device="cuda")
    step = max(1, (1 << 26) // (nb * nb))
    for h in range(c["B"] * c["Hk"]):
        n = s["lens"][h // c["Hk"]]
        m = s["mean"][h].double()
        for a in range(0, c["Nq"], step):
            pos = n - c["Nq"] + torch.arange(a, min(a + step, c["Nq"]), device="cuda")
            score = torch.einsum("gnd,jd->nj", s["q"][h * G:(h + 1) * G, a:a + step].double(), m)
            end = (pos + 1 if c["causal"] else torch.full_like(pos, n))[:, None]
            mine = torch.div(pos, c["block"], rounding_mode="floor")[:, None]
            may = j * c["block"] < end
            must = may & ((j < c["sink"]) | ((j <= mine) & (mine - j < c["local"])))
            free = c["topk"] - must.sum(1, keepdim=True)
            score = torch.where(may & ~must, score, -math.inf)
            beats = (score[:, None, :] > score[:, :, None]) | ((score[:, None, :] == score[:, :, None]) & (j < j[:, None]))
            keep = must | (may & ~must & (beats.sum(2) < free))
            place = keep.cumsum(1) - 1
            row, col = keep.nonzero(as_tuple=True)
            out[h, a + row, place[row, col]] = col.int()
    return out


def _seen(s, h, a, e):
    """Which keys the queries a .. e - 1 of key head h attend: [e - a, Nk]."""
    c = s["case"]
    n = s["lens"][h // c["Hk"]]
    hit = torch.zeros(e - a, _blocks(c) + 1, dtype=torch.bool, device="cuda")
    hit.scatter_(1, torch.where(s["sel"][h, a:e] < 0, _blocks(c), s["sel"][h, a:e]).long(), True)
    hit = hit[:, :-1].repeat_interleave(c["block"], 1)[:, : c["Nk"]]
    key = torch.arange(c["Nk"], device="cuda")
    end = n - c["Nq"] + torch.arange(a, e, device="cuda")[:, None] + 1 if c["causal"] else n
    return hit & (key < end) & (key < n)


def _exact_attend(s):
    c = s["case"]
    G, Nq, D = c["Hq"] // c["Hk"], c["Nq"], c["D"]
    o = torch.zeros(c["B"] * c["Hq"], Nq, D, dtype=torch.float64, device="cuda")
    lse = torch.full(o.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // (c["Nk"] * G))
    for h in range(c["B"] * c["Hk"]):
        q, k, v = s["q"][h * G:(h + 1) * G].double(), s["k"][h].double(), s["v"][h].double()
        for a in range(0, Nq, step):
            e = min(Nq, a + step)
            x = torch.einsum("gnd,md->gnm", q[:, a:e], k) * D ** -0.5
            x = x.masked_fill(~_seen(s, h, a, e), -math.inf)
            z = torch.logsumexp(x, -1)
            lse[h * G:(h + 1) * G, a:e] = z
            o[h * G:(h + 1) * G, a:e] = torch.einsum("gnm,md->gnd", torch.nan_to_num(torch.exp(x - z[..., None])), v)
    return o, lse


def _exact_attend_grad(s):
    c = s["case"]
    G, Nq, Nk, D = c["Hq"] // c["Hk"], c["Nq"], c["Nk"], c["D"]
    dq = torch.zeros(c["B"] * c["Hq"], Nq, D, dtype=torch.float64, device="cuda")
    dk = torch.zeros(c["B"] * c["Hk"], Nk, D, dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)
    step = max(1, (1 << 26) // (Nk * G))
    for h in range(c["B"] * c["Hk"]):
        at = slice(h * G, (h + 1) * G)
        k, v = s["k"][h].double(), s["v"][h].double()
        for a in range(0, Nq, step):
            e = min(Nq, a + step)
            q, do, o = (s[x][at, a:e].double() for x in ("q", "do", "o"))
            p = torch.exp(torch.einsum("gnd,md->gnm", q, k) * D ** -0.5 - s["lse"][at, a:e, None].double())
            p = torch.where(_seen(s, h, a, e), p, 0.0)
            dp = torch.einsum("gnd,md->gnm", do, v)
            ds = p * (dp - torch.einsum("gnd,gnd->gn", do, o)[..., None]) * D ** -0.5
            dq[at, a:e] = torch.einsum("gnm,md->gnd", ds, k)
            dk[h] += torch.einsum("gnm,gnd->md", ds, q)
            dv[h] += torch.einsum("gnm,gnd->md", p, do)
    return dq, dk, dv


_EXACT = {"rope": _exact_rope, "ropegrad": _exact_rope_grad, "mean": _exact_mean, "select": _exact_select,
          "attn": _exact_attend, "attngrad": _exact_attend_grad}


def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s)
