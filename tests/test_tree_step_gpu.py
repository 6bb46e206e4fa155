"""A speculative step as it would be used: store the drafted rows, attend to the
trees, verify, commit, and go on from there; eager and as graphs."""
import numpy as np
import pytest
import torch

from tests import tree_reference as ref
from tests.helpers import bf16_dev_to_bits, dev_to_f64, normal_bits, to_dev_bf16, to_dev_i32

pytestmark = pytest.mark.gpu
SCALE = 1 / np.sqrt(128)
HQ, HKV, V, LAYERS, WIDTH = 6, 2, 300, 2, 12


@pytest.fixture(scope="module")
def ops():
    from paged_kv_continuous_gb300 import ops as o
    return o


class Loop:
    """Three sequences, their pages and counts, and the model's side of every step as seeded
    random rows: K/V and q of the nodes, the target's and the draft's probabilities."""

    def __init__(self, seed, drafts=True):
        self.rng = np.random.default_rng(seed)
        self.drafts = drafts
        self.NB, self.done = 64, np.array([37, 0, 129], np.int32)
        perm = self.rng.permutation(self.NB)
        self.tables = np.full((3, 16), -1, np.int32)
        for b in range(3):  # every sequence has room to grow
            self.tables[b] = perm[16 * b:16 * b + 16]
        self.k = [normal_bits(self.rng, (self.NB, 16, HKV, 128)) for _ in range(LAYERS)]
        self.v = [normal_bits(self.rng, (self.NB, 16, HKV, 128)) for _ in range(LAYERS)]

    def step(self):
        rng = self.rng
        n = rng.integers(0, WIDTH + 1, 3)
        n[rng.integers(3)] = WIDTH
        s = dict(n=n, cu=np.concatenate([[0], np.cumsum(n)]).astype(np.int32))
        T = 3 * WIDTH  # rows of the static buffers; those past cu[3] are not used
        s["parents"] = np.full(T, 77, np.int32)
        s["tokens"] = rng.integers(0, V, T).astype(np.int32)
        s["slots"] = np.full(T, -1, np.int32)
        for b in range(3):
            a = s["cu"][b]
            s["parents"][a:a + n[b]] = ref.random_parents(rng, int(n[b]), 3)
            pos = self.done[b] + np.arange(n[b])
            s["slots"][a:a + n[b]] = self.tables[b, pos // 16] * 16 + pos % 16
        s["ctx"] = (self.done + n).astype(np.int32)
        s["q"] = [normal_bits(rng, (T, HQ, 128)) for _ in range(LAYERS)]
        s["nk"], s["nv"] = ([normal_bits(rng, (T, HKV, 128)) for _ in range(LAYERS)]
                            for _ in range(2))
        z = rng.standard_normal((T, V))
        soft = lambda x: (np.exp(x) / np.exp(x).sum(-1, keepdims=True)).astype(np.float32)
        s["p"] = soft(2 * z)
        s["dq"] = soft(2 * z + 0.5 * rng.standard_normal((T, V))) if self.drafts else None
        for i in range(T):  # likely guesses, so that walks get somewhere
            c = s["parents"][i]
            if 0 <= c < T:
                b = np.searchsorted(s["cu"], i, side="right") - 1
                s["tokens"][i] = np.argsort(-s["p"][s["cu"][b] + c])[rng.integers(3)]
        s["u"], s["ul"] = rng.random(T, np.float32), rng.random(3, np.float32)
        return s

    def reference(self, s):
        """The step's rows, attention and tokens; the pools and lengths after it."""
        outs = []
        for l in range(LAYERS):
            at = s["slots"] >= 0
            self.k[l].reshape(-1, HKV, 128)[s["slots"][at]] = s["nk"][l][at]
            self.v[l].reshape(-1, HKV, 128)[s["slots"][at]] = s["nv"][l][at]
            outs.append(ref.attention(s["q"][l], self.k[l], self.v[l], self.tables, s["ctx"],
                                      s["cu"], s["parents"], SCALE))
        T = s["cu"][-1]
        got = ref.verify_all(s["cu"], s["tokens"], s["parents"], s["p"][:T],
                             None if s["dq"] is None else s["dq"][:T], s["u"], s["ul"], WIDTH)
        ctx = s["ctx"].copy()
        ref.commit(self.k + self.v, self.tables, ctx, s["cu"], got[1], got[0])
        self.done = ctx
        return outs, got


def on_device(s):
    f = lambda x: None if x is None else torch.from_numpy(x).cuda()
    return dict(cu=to_dev_i32(s["cu"]), parents=to_dev_i32(s["parents"]),
                tokens=to_dev_i32(s["tokens"]), slots=to_dev_i32(s["slots"]),
                ctx=to_dev_i32(s["ctx"]), q=[to_dev_bf16(x) for x in s["q"]],
                nk=[to_dev_bf16(x) for x in s["nk"]], nv=[to_dev_bf16(x) for x in s["nv"]],
                p=f(s["p"]), dq=f(s["dq"]), u=f(s["u"]), ul=f(s["ul"]))


def compare(loop, s, outs, tokens, k, v, ctx):
    want, verified = loop.reference(s)
    T = s["cu"][-1]
    for got, (o, a, big) in zip(outs, want):
        bound = ref.attention_bound(o, a, big, SCALE, 256, True)
        assert (np.abs(dev_to_f64(got) - o) <= bound)[:T].all()
    for g, w in zip(tokens, verified):
        assert np.array_equal(g.cpu().numpy(), w)
    for l in range(LAYERS):
        assert np.array_equal(bf16_dev_to_bits(k[l]), loop.k[l])
        assert np.array_equal(bf16_dev_to_bits(v[l]), loop.v[l])
    assert np.array_equal(ctx.cpu().numpy(), loop.done)


@pytest.mark.parametrize("drafts", [True, False])
def test_steps_of_single_calls(ops, drafts):
    loop = Loop(1, drafts)
    k, v = [to_dev_bf16(x) for x in loop.k], [to_dev_bf16(x) for x in loop.v]
    tables, pools = to_dev_i32(loop.tables), ops.PagePools(k + v)
    err, ws = torch.zeros(1, dtype=torch.int32, device="cuda"), ops.tree_workspace()
    for _ in range(6):
        s = loop.step()
        d = on_device(s)
        outs = []
        for l in range(LAYERS):
            ops.store_kv(d["nk"][l], d["nv"][l], k[l], v[l], d["slots"], err, pdl=True)
            outs.append(ops.decode_tree(d["q"][l], d["cu"], d["parents"], k[l], v[l], tables,
                                        d["ctx"], SCALE, WIDTH, workspace=ws, pdl=True))
        tokens = ops.verify_tree(d["tokens"], d["parents"], d["cu"], d["p"], d["u"], d["ul"], WIDTH,
                                 draft_probs=d["dq"], error_flags=err, pdl=True)
        ops.commit_tree(pools, d["cu"], tables, d["ctx"], tokens[1], tokens[0], error_flags=err,
                        pdl=True)
        torch.cuda.synchronize()
        compare(loop, s, outs, tokens, k, v, d["ctx"])
    assert int(err) == 0 and ops.read_error_word(ws) == 0


def test_steps_of_a_graph(ops):
    from paged_kv_continuous_gb300.graph import TreeStepGraph
    loop = Loop(2)
    k, v = [to_dev_bf16(x) for x in loop.k], [to_dev_bf16(x) for x in loop.v]
    refs = torch.zeros(loop.NB, dtype=torch.int32, device="cuda")
    s = loop.step()
    d = on_device(s)
    layers = [dict(q=d["q"][l], k=d["nk"][l], v=d["nv"][l], k_cache=k[l], v_cache=v[l],
                   out=torch.empty_like(d["q"][l])) for l in range(LAYERS)]
    before = [bf16_dev_to_bits(x) for x in k + v]
    g = TreeStepGraph(layers, d["cu"], d["parents"], d["tokens"], to_dev_i32(loop.tables), d["ctx"],
                      d["slots"], SCALE, WIDTH, d["p"], d["u"], d["ul"], draft_probs=d["dq"],
                      ref_counts=refs)
    # making the graph changes neither pools nor lengths
    assert all(np.array_equal(bf16_dev_to_bits(x), b) for x, b in zip(k + v, before))
    assert np.array_equal(g.context_lens.cpu().numpy(), s["ctx"])
    for i in range(5):
        if i:
            s = loop.step()
            e = on_device(s)
            for l in range(LAYERS):
                for name, x in (("q", "q"), ("k", "nk"), ("v", "nv")):
                    layers[l][name].copy_(e[x][l])
            for name in ("p", "dq", "u", "ul"):
                d[name].copy_(e[name])
            g.update(cu_seqlens=e["cu"], parents=e["parents"], tokens=e["tokens"],
                     context_lens=e["ctx"], slot_mapping=e["slots"])
        held = (s["ctx"] + 15) // 16
        for b in range(3):
            refs[to_dev_i32(loop.tables[b, :held[b]]).long()] = 1
        g.replay()
        tokens = g.verify()
        torch.cuda.synchronize()
        compare(loop, s, [x["out"] for x in layers], tokens, k, v, g.context_lens)
        assert int(refs.sum()) == int(((loop.done + 15) // 16).sum())
    assert g.read_error_word() == 0
    with pytest.raises(ops.PagedAttentionError):
        g.update(parents=d["parents"][:-1])


def test_a_chain_step_is_plain_decoding(ops):
    """One node a step, nothing to accept: the rows equal pa_decode's."""
    loop = Loop(3)
    rng = np.random.default_rng(0)
    k, v = to_dev_bf16(loop.k[0]), to_dev_bf16(loop.v[0])
    ctx = to_dev_i32(loop.done + 1)
    q = to_dev_bf16(normal_bits(rng, (3, HQ, 128)))
    cu, par = to_dev_i32([0, 1, 2, 3]), to_dev_i32([-1, -1, -1])
    tables = to_dev_i32(loop.tables)
    a = ops.decode_tree(q, cu, par, k, v, tables, ctx, SCALE, 1, out_dtype=torch.float32)
    b = ops.decode(q, k, v, tables, ctx, SCALE, out_dtype=torch.float32)
    # two kernels, each within the tests' bound of the definition
    bound = 2 * ref.attention_bound(*ref.attention(bf16_dev_to_bits(q), loop.k[0], loop.v[0],
                                                   loop.tables, loop.done + 1, [0, 1, 2, 3],
                                                   np.array([-1] * 3), SCALE), SCALE, 130, False)
    assert (np.abs(dev_to_f64(a) - dev_to_f64(b)) <= bound).all()
