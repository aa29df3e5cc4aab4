"""The operators of a speculative decoding step over the 16-bit paged cache, as a program calls them,
and their plain forms.

The cache: K and V of [pages, Hkv, 64, 128], bf16 or fp16. Three operators work on it:
  append  new tokens' queries and keys are rotated by their positions; rotated keys and values go into
          the pages, rotated queries into rows of their own;
  tree    attention of each sequence's newest tokens, which are the nodes of a tree of drafted tokens (a
          node sees the tokens before the tree, its ancestors and itself) or a chain (causal);
  commit  the path that the model's own tokens confirm is found, and its rows are moved to where the
          sequence goes on.
``run`` computes them in elementary torch operations where ``own`` is false, and calls the library where
it is true.
"""
import math

import torch

own = False

D = 128
PAGE = 64
SM = 1.0 / math.sqrt(D)
VOCAB = 32000
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---- cases ------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of one long sequence, and of a served batch
        dict(name="append_step_b1", op="append", batch=1, lo=1, hi=1, hq=28, hkv=4, at=131000,
             rot=128, interleaved=False, dtype="bf16"),
        dict(name="append_step_b64", op="append", batch=64, lo=1, hi=1, hq=32, hkv=8, at=16000,
             rot=128, interleaved=False, dtype="bf16"),
        # trees of drafted tokens, half of the channels rotated in neighbouring pairs
        dict(name="append_tree_b8", op="append", batch=8, lo=25, hi=61, hq=32, hkv=8, at=9000,
             rot=64, interleaved=True, dtype="fp16"),
        # a long prompt's layer
        dict(name="append_prompt_32k", op="append", batch=1, lo=32768, hi=32768, hq=32, hkv=8, at=0,
             rot=128, interleaved=False, dtype="bf16"),
        # verifying a small tree over a short sequence
        dict(name="tree_4k", op="tree", batch=1, lo=4096, hi=4096, q=12, chain=False, hq=8, hkv=2,
             dtype="bf16", window=0, keep=0),
        # over long sequences together
        dict(name="tree_128k_b4", op="tree", batch=4, lo=131072, hi=131072, q=16, chain=False, hq=28,
             hkv=4, dtype="bf16", window=0, keep=0),
        # a served batch of ragged lengths, larger trees
        dict(name="tree_paged_b8", op="tree", batch=8, lo=5000, hi=16384, q=61, chain=False, hq=32,
             hkv=8, dtype="fp16", window=0, keep=0),
        # over the blocks that a selector kept
        dict(name="tree_masked_128k_b4", op="tree", batch=4, lo=131072, hi=131072, q=25, chain=False,
             hq=28, hkv=4, dtype="bf16", window=0, keep=96),
        # tokens drafted in a row, in a model with a sliding window
        dict(name="draft_window_b32", op="tree", batch=32, lo=4096, hi=16384, q=5, chain=True, hq=32,
             hkv=8, dtype="bf16", window=4096, keep=0),
        # a chunk of a prompt against what is cached already
        dict(name="chunk_2k_at_32k", op="tree", batch=1, lo=32768, hi=32768, q=2048, chain=True,
             hq=32, hkv=8, dtype="bf16", window=0, keep=0),
        # a tree's rows written, and the confirmed path moved into place
        dict(name="commit_b1", op="commit", batch=1, lo=12, hi=12, hkv=4, at=131000, dtype="bf16"),
        dict(name="commit_b64", op="commit", batch=64, lo=25, hi=61, hkv=8, at=16000, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "tree", "tree", "tree", "tree", "commit"])
    dtype = rng.choice(["bf16", "fp16"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.randint(1, 8)
    if op == "append":
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 32768 * 48 // (hkv * (group + 2) * batch)))
        return dict(op=op, batch=batch, lo=rng.randint(max(1, hi // 4), hi), hi=hi, hq=group * hkv,
                    hkv=hkv, at=_log(rng, 1, 250000), rot=rng.choice([128, 128, 64, 32, 96]),
                    interleaved=rng.random() < 0.4, dtype=dtype)
    if op == "commit":
        hi = _log(rng, 1, 256)
        return dict(op=op, batch=_log(rng, 1, 64), lo=rng.randint(max(1, hi // 2), hi), hi=hi, hkv=hkv,
                    at=_log(rng, 1, 250000), dtype=dtype)
    chain = rng.random() < 0.35
    q = rng.choice([_log(rng, 1, 16), _log(rng, 17, 2048)]) if chain else \
        rng.choice([_log(rng, 2, 24), _log(rng, 25, 256)])
    batch = _log(rng, 1, 64 if q <= 16 else 8)
    most = 4 * 131072 * 4 // (hkv * batch)                                     # cached token-heads
    most = min(most, 2048 * 32768 * 32 // (q * batch * group * hkv), 262144)   # (row, key) pairs
    hi = max(q, _log(rng, 64, max(64, most)))
    lo = rng.randint(max(q, hi // 4), hi)
    blocks = (lo + PAGE - 1) // PAGE
    keep = rng.randint(1, blocks) if rng.random() < 0.25 else 0
    window = 0 if keep or rng.random() < 0.7 else rng.randint(1, hi)
    return dict(op="tree", batch=batch, lo=lo, hi=hi, q=q, chain=chain, hq=group * hkv, hkv=hkv,
                dtype=dtype, window=window, keep=keep)


def _spread(lo, hi, count):
    """count whole numbers of [lo, hi], hi among them, in no order."""
    return [hi if b == 0 else lo + (b * 7919 + 13) * 104729 % (hi - lo + 1) for b in range(count)]


def _lens(case):
    """Cached tokens of each sequence (tree), or its new tokens (append, commit)."""
    return _spread(case["lo"], case["hi"], case["batch"])


def _qlens(case):
    """Nodes of each sequence."""
    q = case["q"]
    return [q] * case["batch"] if q == 1 else _spread(max(1, q // 2), q, case["batch"])


def _starts(case):
    """Where each sequence's new tokens go."""
    return [case["at"] * (b + 1) // case["batch"] for b in range(case["batch"])]


def work(case):
    hkv, lens = case["hkv"], _lens(case)
    if case["op"] == "append":
        rows, rotated = sum(lens) * (case["hq"] + 2 * hkv), sum(lens) * (case["hq"] + hkv)
        return {"bytes": rows * 2 * 2 * D, "flops": rotated * 3 * case["rot"]}
    if case["op"] == "commit":  # every row read and written once; about a sixth of them move
        rows = sum(lens) * 2 * hkv
        return {"bytes": rows * 2 * 2 * D, "flops": sum(lens) * hkv * 3 * D}
    hq, window, keep = case["hq"], case["window"], case["keep"]
    keys = pairs = rows = 0
    for n, nq in zip(lens, _qlens(case)):
        rows += nq
        first = n - nq
        if keep:
            blocks = (n + PAGE - 1) // PAGE
            kept = (min(keep, blocks) - 1) * PAGE + n - (blocks - 1) * PAGE
            keys += kept
            pairs += kept * nq
        else:
            keys += min(n, window + nq - 1) if window else n
            for i in range(nq):
                pairs += min(first + i + 1, window) if window else first + i + 1
    return {"bytes": keys * hkv * 2 * 2 * D + rows * hq * (2 * 2 * D + 4), "flops": pairs * hq * 4 * D}


# ---- inputs -----------------------------------------------------------------------------------
def _offsets(counts, dev):
    c = [0]
    for n in counts:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device=dev)


def _normal(shape, gen, dev, dtype):
    return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)


def _tables(first, last, gen, dev):
    """Block table over randomly ordered pages for blocks first[b] .. last[b] of each sequence (other
    entries -1), and the page count."""
    count = [y - x + 1 for x, y in zip(first, last)]
    perm = torch.randperm(sum(count), generator=gen, device=dev).to(torch.int32)
    bt = torch.full((len(count), max(last) + 1), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(count):
        bt[b, first[b]:last[b] + 1] = perm[at:at + n]
        at += n
    return bt, sum(count)


def _trees(counts, seed):
    """Parents (within the sequence, -1 for the first node) and depths of drafted trees: a node hangs
    on one of the few before it."""
    gen = torch.Generator().manual_seed(seed)
    parents, depths = [], []
    for n in counts:
        r = torch.rand(n, generator=gen).tolist()
        depth = [0]
        parents.append(-1)
        for i in range(1, n):
            p = i - 1 - int(r[i] * min(i, 8))
            parents.append(p)
            depth.append(depth[p] + 1)
        depths += depth
    return parents, depths


def _tokens(counts, parents, seed):
    """Drafted tokens, and the model's own token behind each node: often one of its children's."""
    gen = torch.Generator().manual_seed(seed + 1)
    total = sum(counts)
    draft = torch.randint(0, VOCAB, (total,), generator=gen).tolist()
    target = torch.randint(0, VOCAB, (total,), generator=gen).tolist()
    lucky = torch.rand(total, generator=gen).tolist()
    at = 0
    for n in counts:
        for i in range(1, n):
            if lucky[at + i] < 0.6:
                target[at + parents[at + i]] = draft[at + i]
        at += n
    return draft, target


def _frequencies(rot, dev):
    i = torch.arange(rot // 2, device=dev, dtype=torch.float64)
    return (500000.0 ** (-2.0 * i / rot)).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens, hkv, dtype = _lens(case), case["hkv"], DTYPES[case["dtype"]]
    B = case["batch"]
    s = {"case": dict(case)}
    if case["op"] == "tree":
        return _prepare_tree(s, case, seed, gen, dev, lens, hkv, dtype, B)
    hq = case.get("hq", 0)
    starts = _starts(case)
    ends = [x + n for x, n in zip(starts, lens)]
    s["block_table"], pages = _tables([x // PAGE for x in starts], [(x - 1) // PAGE for x in ends], gen,
                                      dev)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    s["cu"] = _offsets(lens, dev)
    # new rows inside the rows of a fused projection
    s["qkv"] = _normal((sum(lens), (hq + 2 * hkv) * D), gen, dev, dtype)
    q, s["k_new"], s["v_new"] = (x.unflatten(-1, (-1, D)) if x.shape[1] else None for x in
                                 s["qkv"].split([hq * D, hkv * D, hkv * D], 1))
    s["q"], s["q_out"] = q, None if q is None else torch.empty(q.shape, dtype=dtype, device=dev)
    s["k"] = _normal((pages, hkv, PAGE, D), gen, dev, dtype)
    s["v"] = _normal((pages, hkv, PAGE, D), gen, dev, dtype)
    s["rot"], s["interleaved"] = case.get("rot", D), case.get("interleaved", False)
    s["inv_freq"] = _frequencies(s["rot"], dev)
    if case["op"] == "commit":
        parents, depths = _trees(lens, seed)
        draft, target = _tokens(lens, parents, seed)
        s["parents"] = torch.tensor(parents, dtype=torch.int32, device=dev)
        s["draft"] = torch.tensor(draft, dtype=torch.int64, device=dev)
        s["target"] = torch.tensor(target, dtype=torch.int64, device=dev)
        s["seq_lens"] = torch.tensor(ends, dtype=torch.int32, device=dev)
        s["path"] = torch.empty_like(s["parents"])
        s["accepted"], s["new_lens"] = torch.empty_like(s["starts"]), torch.empty_like(s["starts"])
        s["next_token"] = torch.empty(B, dtype=torch.int64, device=dev)
        place = [x + d for x, d in zip(_each(starts, lens), depths)]
    elif max(lens) <= 256:
        _, depths = _trees(lens, seed)  # drafted tokens: their places are their depths in the tree
        place = [x + d for x, d in zip(_each(starts, lens), depths)]
    else:
        place = None  # consecutive tokens
    s["rope_positions"] = None if place is None else torch.tensor(place, dtype=torch.int32, device=dev)
    return s


def _each(values, counts):
    return [x for x, n in zip(values, counts) for _ in range(n)]


def _prepare_tree(s, case, seed, gen, dev, lens, hkv, dtype, B):
    hq, qlens = case["hq"], _qlens(case)
    s["block_table"], pages = _tables([0] * B, [(n - 1) // PAGE for n in lens], gen, dev)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["cu"] = _offsets(qlens, dev)
    total = sum(qlens)
    s["parents"] = None
    if not case["chain"]:
        s["parents"] = torch.tensor(_trees(qlens, seed)[0], dtype=torch.int32, device=dev)
    s["qkv"] = _normal((total, (hq + 2 * hkv) * D), gen, dev, dtype)
    s["q"] = s["qkv"][:, :hq * D].unflatten(-1, (hq, D))
    k = _normal((pages, hkv, PAGE, D), gen, dev, dtype)
    # the first tokens and a few others draw attention, as in a trained model
    last = s["q"][s["cu"][1:].long() - 1].float().unflatten(1, (hkv, hq // hkv)).sum(2)
    hat = (6.0 * last / last.norm(dim=-1, keepdim=True)).unsqueeze(2)
    k[s["block_table"][:, 0].long(), :, :4] += hat.to(dtype)
    for i in range(4):
        at = (torch.rand(B, generator=gen, device=dev) * s["seq_lens"]).long()
        page = s["block_table"].gather(1, (at // PAGE)[:, None])[:, 0].long()
        k[page, :, at % PAGE] = hat[:, :, 0].to(dtype)
    s["k"], s["v"] = k, _normal((pages, hkv, PAGE, D), gen, dev, dtype)
    s["keep"] = _mask(case, gen, dev) if case["keep"] else None
    s["out"] = torch.empty((total, hq, D), dtype=dtype, device=dev)
    s["lse"] = torch.empty((total, hq), dtype=torch.float32, device=dev)
    if own:
        import sparse_quantized_attention_gb300 as ffd
        s["params"] = ffd.make_tree_params(
            B, hq, hkv, pages, s["block_table"].shape[1], max_q_len=case["q"], total_q=total,
            q_stride=s["q"].stride(0), dtype=dtype, window=case["window"])
        s["workspace"] = ffd.alloc_tree_workspace(s["params"])
    return s


def _mask(case, gen, dev):
    """A selector's block mask: the first and the newest blocks, and others to the case's count."""
    nb = torch.tensor([(n + PAGE - 1) // PAGE for n in _lens(case)], device=dev)
    most = int(nb.max())
    score = torch.rand((case["batch"], case["hkv"], most), generator=gen, device=dev)
    j = torch.arange(most, device=dev)
    score[:, :, 0] += 2.0
    score += ((j >= nb[:, None] - 17) * 2.0 + (j == nb[:, None] - 1) * 2.0)[:, None]
    score = torch.where((j < nb[:, None])[:, None], score, -1.0)
    mask = torch.zeros_like(score, dtype=torch.uint8)
    top = score.topk(min(case["keep"], most), dim=-1)
    mask.scatter_(2, top.indices, (top.values >= 0).to(torch.uint8))
    return mask


# ---- the operators ----------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        import sparse_quantized_attention_gb300 as ffd
        if op == "tree":
            ffd.ffd_tree_attention(s["params"], s["q"], s["k"], s["v"], s["seq_lens"],
                                   s["block_table"], s["out"], s["workspace"], parents=s["parents"],
                                   cu_q=s["cu"], keep_in=s["keep"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        ffd.ffd_rope_append(s["q"], s["k_new"], s["v_new"], s["inv_freq"], s["starts"],
                            s["block_table"], s["q_out"], s["k"], s["v"], cu_tokens=s["cu"],
                            rope_positions=s["rope_positions"], interleaved=s["interleaved"])
        if op == "append":
            return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
        ffd.ffd_tree_commit(s["draft"], s["target"], s["seq_lens"], s["block_table"], s["k"], s["v"],
                            s["path"], s["accepted"], s["next_token"], s["new_lens"],
                            parents=s["parents"], cu_nodes=s["cu"])
        return {"k": s["k"], "v": s["v"], "path": s["path"], "accepted": s["accepted"],
                "next_token": s["next_token"], "new_lens": s["new_lens"]}
    if op == "tree":
        return _plain_attention(s)
    q = _plain_append(s)
    return {"q": q, "k": s["k"], "v": s["v"]} if op == "append" else _plain_commit(s)


def _token_places(s):
    """Sequence, place within it and cache token of every new row."""
    cu = s["cu"].long()
    t = torch.arange(s["k_new"].shape[0], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, t - cu[b], s["starts"].long()[b] + t - cu[b]


def _plain_append(s):
    """Angles in 64 bits (far positions), the rotation in 32."""
    b, _, token = _token_places(s)
    place = token if s["rope_positions"] is None else s["rope_positions"].long()
    angle = place.double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    rot, half = s["rot"], s["rot"] // 2

    def turned(x):
        f = x.float()
        if s["interleaved"]:
            a, c = f[..., 0:rot:2], f[..., 1:rot:2]
            y = torch.stack((a * cos - c * sin, a * sin + c * cos), -1).flatten(-2)
        else:
            a, c = f[..., :half], f[..., half:rot]
            y = torch.cat((a * cos - c * sin, a * sin + c * cos), -1)
        return torch.cat((y, f[..., rot:]), -1).to(x.dtype)

    page, row = s["block_table"].long()[b, token // PAGE], token % PAGE
    s["k"][page, :, row] = turned(s["k_new"])
    s["v"][page, :, row] = s["v_new"]
    return None if s["q"] is None else turned(s["q"])


def _padded(s, q):
    """Place of each node in the padded batch [B, q], and the nodes' number in each sequence."""
    cu = s["cu"].long()
    t = torch.arange(s["parents"].shape[0] if s["parents"] is not None else s["q"].shape[0],
                     device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, t - cu[b], cu[1:] - cu[:-1]


def _ancestors(parents, b, i, B, q):
    """[B, q, q]: whether u is i or an ancestor of i. The relation is squared until it reaches the depth
    of any tree that may be given (256 nodes)."""
    step = torch.eye(q, device=parents.device).repeat(B, 1, 1)
    has = parents >= 0
    step[b, i, parents.long().clamp(min=0)] = torch.maximum(
        step[b, i, parents.long().clamp(min=0)], has.float())
    for _ in range(8):
        step = ((step @ step) > 0).float()
    return step > 0


def _visible(s, width):
    """Which of `width` keys each row of the padded batch sees [B, Hkv, q, width], and the place of
    each node in the padded batch."""
    case = s["case"]
    B, q = case["batch"], case["q"]
    b, i, nq = _padded(s, q)
    first = s["seq_lens"].long() - nq
    j = torch.arange(width, device=first.device)
    u = j - first[:, None]                                     # [B, width]: node of a key
    before = (u < 0)[:, None]
    at = u.clamp(0, q - 1)
    r = torch.arange(q, device=first.device)
    if s["parents"] is None:
        depth = r.expand(B, q)
        see = u[:, None] <= r[:, None]
    else:
        anc = _ancestors(s["parents"], b, i, B, q)
        depth = anc.sum(-1) - 1
        see = before | anc.gather(2, at[:, None].expand(-1, q, -1))
    see = see & ((u < nq[:, None])[:, None] & (r < nq[:, None])[:, :, None])
    if case["window"]:
        place = torch.where(u < 0, u, depth.gather(1, at))     # counted from the tree's root
        see &= place[:, None] > depth[:, :, None] - case["window"]
    see = see[:, None].expand(-1, case["hkv"], -1, -1)
    if case["keep"]:
        see = see & (s["keep"] != 0).repeat_interleave(PAGE, -1)[:, :, None, :width]
    return see, b, i


def _plain_attention(s):
    case = s["case"]
    hkv, group, q = case["hkv"], case["hq"] // case["hkv"], case["q"]
    bt = s["block_table"].long().clamp(min=0)
    see, b, i = _visible(s, bt.shape[1] * PAGE)
    # [B, Hkv, keys, 128] of the padded batch
    k, v = (s[x][bt].transpose(1, 2).flatten(2, 3).float() for x in ("k", "v"))
    qp = torch.zeros((case["batch"], q, case["hq"], D), device=k.device)
    qp[b, i] = s["q"].float()
    qp = qp.unflatten(2, (hkv, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)     # [B, Hkv, q G, 128]
    sc = ((qp @ k.transpose(-1, -2)) * SM).unflatten(2, (q, group))
    sc = sc.masked_fill(~see[:, :, :, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(sc - m)
    l = p.sum(-1, keepdim=True)
    out = (p.flatten(2, 3) @ v).unflatten(2, (q, group)) / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m + torch.log(l))[..., 0]
    out = out.permute(0, 2, 1, 3, 4).flatten(2, 3)[b, i]
    return {"out": out.to(s["out"].dtype), "lse": lse.permute(0, 2, 1, 3).flatten(2, 3)[b, i]}


def _plain_commit(s):
    B, q = s["case"]["batch"], s["case"]["hi"]
    b, i, nq = _padded(s, q)
    parents = s["parents"].long()
    up = (s["cu"].long()[b] + parents).clamp(min=0)            # row of the parent
    ok = (i == 0) | ((parents >= 0) & (s["draft"] == s["target"][up]))
    anc = _ancestors(s["parents"], b, i, B, q)
    refused = torch.zeros((B, q), device=parents.device)
    refused[b, i] = (~ok).float()
    r = torch.arange(q, device=parents.device)
    taken = ((anc.float() * refused[:, None]).sum(-1) == 0) & (r < nq[:, None])
    depth = anc.sum(-1) - 1
    # the deepest taken node, the lowest of several
    end = torch.where(taken, depth * q + (q - 1 - r), -1).argmax(-1)
    on = anc.gather(1, end[:, None, None].expand(-1, 1, q))[:, 0]
    accepted = on.sum(-1)
    rank = torch.where(on, on.long().cumsum(-1) - 1, q)
    path = torch.full((B, q + 1), -1, device=parents.device).scatter(1, rank, r.expand(B, q))[:, :q]
    first = s["seq_lens"].long() - nq
    # rows behind the path stay; padded ones are the last node's
    stay = torch.minimum(r.expand(B, q), nq[:, None] - 1)
    to, source = first[:, None] + stay, first[:, None] + torch.where(path >= 0, path, stay)
    pages = s["block_table"].long()
    from_page, to_page = pages.gather(1, source // PAGE), pages.gather(1, to // PAGE)
    rows_k, rows_v = (s[x][from_page, :, source % PAGE] for x in ("k", "v"))
    s["k"][to_page, :, to % PAGE] = rows_k
    s["v"][to_page, :, to % PAGE] = rows_v
    last = s["cu"].long()[:-1] + end
    return {"k": s["k"], "v": s["v"], "path": path[b, i].to(torch.int32),
            "accepted": accepted.to(torch.int32), "next_token": s["target"][last],
            "new_lens": (first + accepted).to(torch.int32)}


# ---- the definition in 64 bits ----------------------------------------------------------------
def _turned64(x, place, s):
    """Rows x [T, heads, 128] in 64 bits, pair by pair."""
    y = x.to(torch.float64).clone()
    half = s["rot"] // 2
    for p in range(half):
        a, c = (2 * p, 2 * p + 1) if s["interleaved"] else (p, p + half)
        turn = (place.to(torch.float64) * s["inv_freq"][p].to(torch.float64))[:, None]
        xa, xc = x[..., a].to(torch.float64), x[..., c].to(torch.float64)
        y[..., a] = torch.cos(turn) * xa - torch.sin(turn) * xc
        y[..., c] = torch.sin(turn) * xa + torch.cos(turn) * xc
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_attention(case, s)
    lens, starts, bt = _lens(case), _starts(case), s["block_table"].long()
    place = s["rope_positions"]
    if place is None:
        place = torch.cat([torch.arange(x, x + n, device=bt.device) for x, n in zip(starts, lens)])
    k, v = s["k"].to(torch.float64), s["v"].to(torch.float64)
    rows, at = _turned64(s["k_new"], place, s), 0
    for b, (start, n) in enumerate(zip(starts, lens)):
        t = torch.arange(start, start + n, device=bt.device)
        k[bt[b, t // PAGE], :, t % PAGE] = rows[at:at + n]
        v[bt[b, t // PAGE], :, t % PAGE] = s["v_new"][at:at + n].to(torch.float64)
        at += n
    if case["op"] == "append":
        return {"q": _turned64(s["q"], place, s), "k": k, "v": v}
    draft, target, parents = (s[x].tolist() for x in ("draft", "target", "parents"))
    table, at = bt.tolist(), 0
    for b, (start, n) in enumerate(zip(starts, lens)):
        best, chosen = -1, []
        for i in range(n):
            chain, u = [i], i
            while parents[at + u] >= 0:
                u = parents[at + u]
                chain.append(u)
            chain.reverse()
            fits = chain[0] == 0 and all(draft[at + y] == target[at + x] for x, y in zip(chain, chain[1:]))
            if fits and len(chain) > best:
                best, chosen = len(chain), chain
        for to, node in enumerate(chosen):  # ascending: what is read has not been written yet
            x, y = start + node, start + to
            k[table[b][y // PAGE], :, y % PAGE] = k[table[b][x // PAGE], :, x % PAGE].clone()
            v[table[b][y // PAGE], :, y % PAGE] = v[table[b][x // PAGE], :, x % PAGE].clone()
        at += n
    return {"k": k, "v": v, "path": None, "accepted": None, "next_token": None, "new_lens": None}


def _exact_attention(case, s):
    lens, bt, hkv, dev = _lens(case), s["block_table"].long(), case["hkv"], s["block_table"].device
    group, at, outs, lses = case["hq"] // hkv, 0, [], []
    for b, (n, nq) in enumerate(zip(lens, _qlens(case))):
        pages = bt[b, :(n + PAGE - 1) // PAGE]
        first = n - nq
        hidden = torch.zeros((nq, n), dtype=torch.bool, device=dev)
        place = torch.arange(n, device=dev)  # of each key
        if s["parents"] is None:
            hidden[:, first:] = torch.ones((nq, nq), dtype=torch.bool, device=dev).triu(1)
        else:
            up = s["parents"][at:at + nq].tolist()
            mine, depth = torch.zeros((nq, nq), dtype=torch.bool), []
            for i, p in enumerate(up):
                if p >= 0:
                    mine[i] = mine[p]
                mine[i, i] = True
                depth.append(depth[p] + 1 if p >= 0 else 0)
            hidden[:, first:] = ~mine.to(dev)
            place[first:] = first + torch.tensor(depth, device=dev)
        if case["window"]:
            hidden |= place[None] <= place[first:, None] - case["window"]
        o = torch.empty((nq, case["hq"], D), dtype=torch.float64, device=dev)
        z = torch.empty((nq, case["hq"]), dtype=torch.float64, device=dev)
        for h in range(hkv):
            k, v = (s[x][pages, h].to(torch.float64).flatten(0, 1)[:n] for x in ("k", "v"))
            unseen = hidden
            if case["keep"]:
                unseen = hidden | (s["keep"][b, h].repeat_interleave(PAGE)[:n] == 0)[None]
            for g in range(group):
                x = (s["q"][at:at + nq, h * group + g].to(torch.float64) @ k.T) / math.sqrt(D)
                x[unseen] = -math.inf
                z[:, h * group + g] = torch.logsumexp(x, -1)
                empty = unseen.all(-1, keepdim=True)
                p = torch.where(empty, 0.0, torch.softmax(x, -1))
                o[:, h * group + g] = p @ v
        at += nq
        outs.append(o)
        lses.append(z)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
