"""The cache's operators in a run, as a decoder uses them: a small GPT-2-shaped
model with 4-bit weights and the int8 head, prompts of unequal length attended
causally, token by token decoding with scores read from the logits, and an
eviction on the way; against the same model in fp64 on the CPU.

Bound of the logits: every matmul of the model is within 1e-5 sum |x w|, which
for sums of 128 to 256 terms of random sign is at most about 1.5e-4 of their
result's size; nine of them, and the attention's and norms' roundings below
that, one behind the other: 2e-3 of the largest logit."""

import numpy as np
import pytest

import oracle
from kv_util import clear_error, error_status, read_rows, torch, w4

pytestmark = pytest.mark.gpu

E, H, D, LAYERS, V, MLP, PAGE = 128, 2, 64, 2, 1003, 256, 16


class Model:
    """Weights on the GPU and, dequantised, in fp64."""

    def __init__(self, seed):
        T, W = torch(), w4()
        rng = np.random.default_rng(seed)
        table = rng.integers(-127, 128, (E, V)).astype(np.int8)
        self.scales = (rng.random(V) * 0.004 + 0.002).astype(np.float32)
        self.table, self.emb = table, table.astype(np.float64) * self.scales
        self.td, self.sd = T.from_numpy(table).cuda(), T.from_numpy(self.scales).cuda()
        self.tiles = W.i8t_head_repack(self.td, self.sd, E, V)
        self.layers = []
        for _ in range(LAYERS):
            layer = {}
            for name, k, n in (("qkv", E, 3 * E), ("proj", E, E), ("fc", E, MLP), ("out", MLP, E)):
                w = (rng.standard_normal((k, n)) * 0.08).astype(np.float32)
                b = (rng.standard_normal(n) * 0.02).astype(np.float32)
                qw, sc, zp = W.w4_quantize(T.from_numpy(w).cuda())
                wt = W.w4t_repack(qw, sc, zp, k, n)
                eye, _ = oracle.w4_matmul_ref(np.eye(k, dtype=np.float32), qw.cpu().numpy(), sc.cpu().numpy(),
                                              zp.cpu().numpy(), k, n)
                layer[name] = (wt, k, n, T.from_numpy(b).cuda(), np.asarray(eye), b.astype(np.float64))
            self.layers.append(layer)


def norm(x):
    return torch().nn.functional.layer_norm(x, (E,))


def norm64(x):
    return (x - x.mean(-1, keepdims=True)) / np.sqrt(x.var(-1, keepdims=True) + 1e-5)


def linear(x, w, **kw):
    return w4().w4t_matmul(x, w[0], w[1], w[2], bias=w[3], **kw)


def forward(m, caches, x, append, attend):
    """x [rows, E] through the layers; append and attend as the phase needs them."""
    for layer, cache in zip(m.layers, caches):
        qkv = linear(norm(x), layer["qkv"])
        heads = [qkv[:, i * E:(i + 1) * E].view(-1, H, D) for i in range(3)]
        append(cache, heads[1], heads[2])
        x = linear(attend(cache, heads[0]).view(-1, E), layer["proj"], residual=x)
        x = linear(linear(norm(x), layer["fc"], act="gelu_tanh"), layer["out"], residual=x)
    return norm(x)


def forward64(m, slots, token):
    """One token of one sequence in fp64; slots[layer] = (keys, values) so far, extended."""
    x = m.emb[:, token]
    weights = []
    for layer, kv in zip(m.layers, slots):
        def lin(v, name):
            return v @ layer[name][4] + layer[name][5]
        q, k, v = (y.reshape(H, D) for y in np.split(lin(norm64(x), "qkv"), 3))
        kv[0].append(k)
        kv[1].append(v)
        out, _, w, _ = oracle.kv_attend_ref(q, np.stack(kv[0]), np.stack(kv[1]), D ** -0.5)
        weights.append(w.sum(0))
        x = x + lin(out.reshape(-1), "proj")
        h = lin(norm64(x), "fc")
        h = 0.5 * h * (1 + np.tanh(np.sqrt(2 / np.pi) * (h + 0.044715 * h ** 3)))
        x = x + lin(h, "out")
    return norm64(x) @ m.emb, weights


def test_prompts_decoding_and_eviction():
    T, W = torch(), w4()
    clear_error()
    m = Model(5)
    rng = np.random.default_rng(6)
    lens, steps, room = [5, 1, 19], 24, 48
    B = len(lens)
    tokens = [rng.integers(0, V, n + steps) for n in lens]
    table = T.from_numpy(rng.permutation(B * room // PAGE).reshape(B, -1).astype(np.int32)).cuda()
    caches = [W.KvCache.empty(B * room // PAGE, H, PAGE, D, table, T.float32) for _ in range(LAYERS)]
    accs = [T.zeros((B, room), device="cuda") for _ in range(LAYERS)]
    slots = [[([], []) for _ in range(LAYERS)] for _ in range(B)]
    sums = [[np.zeros(0) for _ in range(LAYERS)] for _ in range(B)]
    cu = T.tensor(np.r_[0, np.cumsum(lens)], dtype=T.int32, device="cuda")

    def embed(ids):
        return W.i8_embed_lookup(m.td, m.sd, T.tensor(np.asarray(ids), dtype=T.int32, device="cuda"), E, V)

    # the prompts: all tokens enter the caches, each attends its sequence up to itself
    def attend_prompt(cache, q):
        out = []
        for b, n in enumerate(lens):
            rows = W.KvCache(cache.k, cache.v, cache.page_table[b:b + 1].expand(n, -1),
                             T.arange(1, n + 1, dtype=T.int32, device="cuda"))
            a = T.zeros((n, room), device="cuda")
            out.append(W.kv_attend(q[cu[b]:cu[b + 1]], rows, acc=a))
            accs[caches.index(cache)][b] += a.sum(0)
        return T.cat(out)

    x = forward(m, caches, embed(np.concatenate([t[:n] for t, n in zip(tokens, lens)])),
                lambda c, k, v: W.kv_append(c, k, v, cu_tokens=cu), attend_prompt)
    h = x[(cu[1:] - 1).long()]
    for b, n in enumerate(lens):
        for t in tokens[b][:n]:
            want, weights = forward64(m, slots[b], t)
            sums[b] = [np.append(s, 0.0) + w for s, w in zip(sums[b], weights)]
        slots[b].append(want)  # the logits behind the prompt
    want = np.stack([s.pop() for s in slots])

    for step in range(steps):
        logits = W.i8t_head_logits(h, m.tiles, E, V)
        nxt = np.array([t[n + step] for t, n in zip(tokens, lens)], np.int32)
        logp, ent, tl, ti = W.token_logprobs(logits, T.from_numpy(nxt).cuda(), top=3)
        tol = 2e-3 * np.abs(want).max()
        assert np.abs(logits.cpu().numpy() - want).max() <= tol, step
        rp, re, rtl, _ = oracle.logprobs_ref(want, nxt, 3)
        assert np.abs(logp.cpu().numpy() - rp).max() <= 2 * tol and np.abs(tl.cpu().numpy() - rtl).max() <= 2 * tol
        spread = np.abs(want - want.max(1, keepdims=True)).max()
        assert np.abs(ent.cpu().numpy() - re).max() <= 2 * tol * (1 + spread)
        assert np.array_equal(ti[:, 0].cpu().numpy(), W.i8t_head_argmax(h, m.tiles, E, V)[0].cpu().numpy())
        if step == 12:  # every layer's cache is cut to the 14 slots its own attention used most
            for i, (cache, acc) in enumerate(zip(caches, accs)):
                before, a = cache.lengths.tolist(), acc.cpu().numpy().copy()
                kept = T.zeros((B, 14), dtype=T.int32, device="cuda")
                W.kv_evict(cache, acc, 14, recent=4, kept=kept)
                for b in range(B):
                    assert np.abs(a[b, :before[b]] - sums[b][i]).max() <= 2e-3 * before[b]
                    j = oracle.kv_evict_ref(a[b], before[b], 14, 4)
                    assert kept[b, :len(j)].tolist() == j
                    slots[b][i] = tuple([s[k] for k in j] for s in slots[b][i])
                    sums[b][i] = sums[b][i][j]
            assert caches[0].lengths.tolist() == [14, 13, 14]
        by_layer = iter(accs)
        h = forward(m, caches, embed(nxt), lambda c, k, v: W.kv_append(c, k, v),
                    lambda c, q: W.kv_attend(q, c, acc=next(by_layer)))
        want = []
        for b in range(B):
            w, weights = forward64(m, slots[b], int(nxt[b]))
            want.append(w)
            sums[b] = [np.append(s, 0.0) + x for s, x in zip(sums[b], weights)]
        want = np.stack(want)
    for cache, i in zip(caches, range(LAYERS)):
        for b in range(B):
            gk, gv = read_rows(cache, b, len(slots[b][i][0]))
            assert np.abs(gk - np.stack(slots[b][i][0])).max() <= 2e-2
    assert error_status() == 0


@pytest.mark.parametrize("dtype", ["float32", "int8"])
def test_a_captured_step_decodes_as_the_eager_one(dtype):
    """The whole step in a graph (embedding, layers, head, scores), replayed
    while the cache fills: bit for bit the eager step's results."""
    T, W = torch(), w4()
    m = Model(9)
    rng = np.random.default_rng(10)
    B, room, steps = 3, 48, 40
    ids = T.zeros(B, dtype=T.int32, device="cuda")
    runs = []
    for _ in range(2):
        table = T.arange(B * room // PAGE, dtype=T.int32, device="cuda").view(B, -1)
        runs.append([W.KvCache.empty(B * room // PAGE, H, PAGE, D, table, getattr(T, dtype)) for _ in range(LAYERS)])

    def step(caches):
        x = W.i8_embed_lookup(m.td, m.sd, ids, E, V)
        h = forward(m, caches, x, lambda c, k, v: W.kv_append(c, k, v), lambda c, q: W.kv_attend(q, c))
        return W.token_logprobs(W.i8t_head_logits(h, m.tiles, E, V), ids, top=4)

    step(runs[0])
    for c in runs[0]:
        c.lengths.zero_()
    T.cuda.synchronize()
    g = T.cuda.CUDAGraph()
    with T.cuda.graph(g):
        captured = step(runs[0])
    for _ in range(steps):
        ids.copy_(T.from_numpy(rng.integers(0, V, B).astype(np.int32)))
        g.replay()
        eager = step(runs[1])
        T.cuda.synchronize()
        assert all(T.equal(a, b) for a, b in zip(captured, eager))
    assert runs[0][0].lengths.tolist() == [steps] * B
