"""cb_paged_attention_shared: host validation (CPU) and, on the GPU, the shared form against the
float64 oracle and the plain step."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_kv_attention_cb_gb300 as cb
import workloads
from paged_kv_attention_cb_gb300 import build as cbbuild

FAKE = 0x100000


@pytest.fixture(scope="module")
def lib():
    cbbuild.build()
    return cb.lib()


def call(lib, qsl, seq, prefix, groups, *, BS=16, Hq=4, Hkv=2, D=64, dtype=1, ws_bytes=None, plen=FAKE,
         out=FAKE, mirrors=True):
    qsl, seq, prefix, groups = (np.ascontiguousarray(a, np.int32) for a in (qsl, seq, prefix, groups))
    R, T = len(seq), int(qsl[-1])
    stride = max(1, int(max((seq + BS - 1) // BS)))
    if ws_bytes is None:
        ws_bytes = lib.cb_workspace_size_shared(R, T, Hq, Hkv, D)
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    return lib.cb_paged_attention_shared(out, FAKE, FAKE, FAKE, None, None, None, FAKE, FAKE, FAKE, stride, plen,
                                         p(qsl), p(seq), p(prefix) if mirrors else None,
                                         p(groups) if mirrors else None, len(groups) - 1, R, T, 40, BS, Hq, Hkv, D,
                                         0.0, 0, dtype, 0, FAKE, ws_bytes, None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(prefix=[32, 16]), 2),                          # lengths differ within a group
    (dict(prefix=[24, 24]), 2),                          # not whole blocks
    (dict(prefix=[48, 48], seq=[48, 60]), 2),            # reaches into the step's own tokens
    (dict(prefix=[-16, -16]), 2),
    (dict(qsl=[0, 2, 3], prefix=[32, 32]), 2),           # a run of tokens cannot share
    (dict(groups=[0, 1]), 2), (dict(groups=[1, 2]), 2), (dict(groups=[0, 2, 1, 2]), 2), (dict(groups=[0, 3, 2]), 2),
    (dict(mirrors=False), 1), (dict(plen=None), 1), (dict(out=None), 1),
    (dict(ws_bytes=1000), 4), (dict(D=96), 3), (dict(qsl=[0, 1, 1], seq=[50, -1]), 2),
])
def test_refusals(lib, kwargs, status):
    base = dict(qsl=[0, 1, 2], seq=[50, 60], prefix=[32, 32], groups=[0, 2])
    assert call(lib, **{**base, **kwargs}) == status
    assert lib.cb_last_error_message()


def test_nothing_to_do(lib):
    assert call(lib, [0, 0, 0], [50, 60], [32, 32], [0, 2]) == 0


# ------------------------------------------------------------------ on the GPU


def shared_spec(groups, *, block_size=16, seed=0, extra_q=(), **kw):
    """groups: (prefix length, [suffix length of each request, this step's token included; 0: a
    request without tokens]). extra_q: (q_len, ctx) of requests that follow, sharing nothing."""
    q, ctx, pre, start = [], [], [], [0]
    for p, suf in groups:
        for s in suf:
            q.append(1 if s else 0)
            ctx.append(p + max(s, 1) - 1)
            pre.append(p)
        start.append(len(q))
    for a, b in extra_q:
        q.append(a)
        ctx.append(b)
        pre.append(0)
        start.append(len(q))
    spec = workloads.custom(q, ctx, block_size=block_size, seed=seed, pool_factor=1.3, **kw)
    r = 0
    for p, suf in groups:
        for i in range(1, len(suf)):
            spec = workloads.share_prefix_pages(spec, r, r + i, p // block_size)
        r += len(suf)
    return spec, np.array(pre, np.int32), np.array(start, np.int32)


class Step:
    def __init__(self, groups, **kw):
        self.spec, self.prefix, self.start = shared_spec(groups, **kw)
        s = self.spec
        self.x = workloads.draw_tensors(s, "cuda")
        self.md = workloads.metadata_tensors(s, "cuda")
        self.plen = torch.from_numpy(self.prefix).cuda()
        self.ws = cb.alloc_workspace_shared(s.R, s.T, s.num_q_heads, s.num_kv_heads, s.head_dim)
        self.before = {k: v.clone() for k, v in self.x.items()}

    def run(self, flags=cb.CB_FLAG_SHARE_ALWAYS, out=None, ws=None):
        s, x = self.spec, self.x
        if out is None:
            out = torch.full_like(x["q"], float("nan"))
        return cb.paged_attention_shared(
            out, x["q"], x["k_cache"], x["v_cache"], self.md["query_start_loc"], self.md["seq_lens"],
            self.md["block_table"], self.plen, s.query_start_loc, s.seq_lens, self.prefix, self.start,
            self.ws if ws is None else ws, scale=s.scale, sliding_window=s.sliding_window, k_new=x["k_new"],
            v_new=x["v_new"], slot_mapping=self.md["slot_mapping"], flags=flags)

    def check(self, out):
        """Weights are rounded to bf16 (2^-8 of themselves, after a score error of 2^-16 of the sum
        of its products' magnitudes), sums over n keys are fp32 (n 2^-23), outputs bf16 (2^-8)."""
        s = self.spec
        h = {k: v.double().cpu().numpy() for k, v in self.before.items()}
        ref, kc, vc = oracle.step(h["q"], h["k_cache"], h["v_cache"], h["k_new"], h["v_new"], s.slot_mapping,
                                  s.query_start_loc, s.seq_lens, s.block_table, s.block_size, s.scale,
                                  s.sliding_window)
        absv = oracle.paged_attention(h["q"], kc, np.abs(vc), s.query_start_loc, s.seq_lens, s.block_table,
                                      s.block_size, s.scale, s.sliding_window)
        G = s.num_q_heads // s.num_kv_heads
        B = s.scale * (np.abs(h["q"]).reshape(s.T, s.num_kv_heads, G, -1)
                       * np.abs(kc).max(axis=(0, 1))[None, :, None]).sum(-1).reshape(s.T, s.num_q_heads, 1)
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -15 * B + 2.0 ** -8 + int(s.seq_lens.max()) * 2.0 ** -23) * absv
        got = out.double().cpu().numpy()
        assert np.isfinite(got).all()
        assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())
        assert np.array_equal(self.x["k_cache"].double().cpu().numpy(), kc)
        assert np.array_equal(self.x["v_cache"].double().cpu().numpy(), vc)


def prefix_launches():
    return cb.launch_count(cb.kernel_names().index("prefix_tc"))


GROUPS = [
    [(64, [1, 5])],
    [(16, [1])],
    [(128, [1, 16, 17, 0, 40])],
    [(144, [3] * 33)],
    [(0, [30, 7]), (2048, [100, 1, 33]), (0, [200])],
    [(256, [9] * 5), (640, [1, 300]), (16, [20, 2, 2]), (1008, [64] * 70)],
]


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,BS", [(32, 8, 128, 16), (8, 8, 64, 8), (16, 1, 128, 16), (32, 16, 64, 16),
                                         (4, 4, 128, 8), (10, 5, 128, 16), (16, 4, 64, 16)])
@pytest.mark.parametrize("case", range(len(GROUPS)))
def test_shared_against_oracle(case, Hq, Hkv, D, BS):
    st = Step(GROUPS[case], num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, block_size=BS, seed=case)
    n = prefix_launches()
    out = st.run()
    st.check(out)
    assert prefix_launches() == n + 1
    assert cb.read_error_word(st.ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("BS,P", [(32, 96), (64, 640), (128, 384), (256, 512)])
def test_larger_pages(BS, P):
    st = Step([(P, [1, 40, 3]), (BS, [5, 5])], block_size=BS, seed=3)
    st.check(st.run())


@pytest.mark.gpu
def test_beside_runs_of_tokens():
    """Chunks in the same step: the prefix of the decode rows, the chunks by themselves."""
    st = Step([(320, [4, 50, 1])], extra_q=[(130, 0), (1, 90), (40, 200), (3, 3)], seed=5)
    n = prefix_launches()
    st.check(st.run())
    assert prefix_launches() == n + 1


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(dtype="f32"), dict(sliding_window=100), dict(block_size=4)])
def test_plain_forms(kw):
    """What the shared form does not cover runs as the plain step."""
    st = Step([(128, [4, 50, 1])], num_q_heads=8, num_kv_heads=2, seed=6, **kw)
    n = prefix_launches()
    st.check(st.run())
    assert prefix_launches() == n


@pytest.mark.gpu
def test_small_groups_run_plainly():
    st = Step([(64, [4, 9])], seed=6)
    n = prefix_launches()
    st.check(st.run(flags=0))
    assert prefix_launches() == n


@pytest.mark.gpu
def test_no_groups_is_the_plain_step():
    st = Step([(64, [4, 9])], seed=6)
    st.start = np.zeros(1, np.int32)
    st.check(st.run())


@pytest.mark.gpu
def test_long_prefix_agrees_with_the_plain_step():
    st = Step([(16384, [5 + 7 * i for i in range(24)]), (4096, [300] * 20)], seed=7)
    out = st.run(flags=0)
    s, x = st.spec, st.x
    plain = torch.empty_like(out)
    cb.paged_attention(plain, x["q"], x["k_cache"], x["v_cache"], st.md["query_start_loc"], st.md["seq_lens"],
                       st.md["block_table"], s.query_start_loc, s.seq_lens,
                       cb.alloc_workspace(s.R, s.T, s.num_q_heads, s.num_kv_heads, s.head_dim), scale=s.scale)
    # each is within bf16 weights and outputs of the same value: 2^-8 of it and of |V| (max ~5) / sqrt(n)
    d = (out.float() - plain.float()).abs()
    assert d.max() <= 2 * (2.0 ** -8 * plain.float().abs().max() + 2.0 ** -8)
    rows = [0, 11, 23, 24, 43]
    h = {k: v.double().cpu().numpy() for k, v in st.before.items()}
    oracle.scatter_kv(h["k_cache"], h["v_cache"], h["k_new"], h["v_new"], s.slot_mapping)
    ref = oracle.paged_attention(h["q"], h["k_cache"], h["v_cache"], s.query_start_loc, s.seq_lens, s.block_table,
                                 s.block_size, s.scale, rows=rows)
    got = out.double().cpu().numpy()[rows]
    assert np.abs(got - ref[rows]).max() <= 2.0 ** -8 * (np.abs(ref[rows]).max() + 1)


@pytest.mark.gpu
def test_a_workspace_serves_steps_of_any_size_and_replays():
    ws = cb.alloc_workspace_shared(80, 400, 32, 8, 128)
    for groups, extra in (([(512, [3] * 70)], []), ([(64, [1, 2])], [(300, 100)]), ([(2048, [40, 3, 9])], [])):
        st = Step(groups, extra_q=extra, seed=len(groups[0][1]))
        st.check(st.run(ws=ws))
    assert cb.read_error_word(ws) == 0
    st = Step([(512, [3] * 40), (1024, [70, 2])], seed=1)
    out = st.run().clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        st.run()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    buf = torch.empty_like(out)
    with torch.cuda.graph(g):
        st.run(out=buf)
    for _ in range(3):
        buf.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, out)
    st.check(buf)


@pytest.mark.gpu
def test_addresses_aligned_to_sixteen_bytes():
    def shifted(t):
        flat = torch.empty(t.numel() + 16 // t.element_size(), dtype=t.dtype, device=t.device)
        return flat[16 // t.element_size():].view(t.shape).copy_(t)

    st = Step([(512, [3] * 40), (1024, [70, 2])], extra_q=[(300, 100)], seed=1)
    st.x = {k: shifted(v) for k, v in st.x.items()}
    st.ws = shifted(st.ws)
    before = prefix_launches()
    st.check(st.run(out=shifted(torch.full_like(st.x["q"], float("nan")))))
    assert prefix_launches() == before + 1


@pytest.mark.gpu
def test_bad_prefix_page_is_recorded():
    st = Step([(256, [3, 9])], seed=2)
    st.md["block_table"][0, 3] = st.spec.num_blocks + 1
    out = st.run()
    assert torch.isfinite(out.float()).all()
    assert cb.read_error_word(st.ws) == cb.CB_DEVERR_BLOCK_ID


@pytest.mark.gpu
def test_a_wait_that_runs_out_is_reported():
    st = Step([(512, [30, 9, 100])], seed=2)
    st.run(flags=cb.CB_FLAG_SHARE_ALWAYS | cb.CB_FLAG_TEST_WAIT_EXPIRY)
    assert cb.read_error_word(st.ws) & cb.CB_DEVERR_TIMEOUT
    cb.workspace_init(st.ws)
    for k in st.x:
        st.x[k].copy_(st.before[k])
    st.check(st.run())


@pytest.mark.gpu
def test_binding_refuses():
    st = Step([(64, [4, 9])], seed=6)
    good = st.plen
    for bad in (good.long(), good[:1], good.cpu()):
        st.plen = bad
        with pytest.raises(cb.CbError):
            st.run()
    st.plen = good
    st.prefix = st.prefix + 8
    with pytest.raises(cb.CbError):
        st.run()


@pytest.mark.gpu
def test_samples_of_one_prompt_step_by_step():
    """A prompt is prefilled once; five requests share its whole blocks and decode tokens of their
    own, each step writing its rows and attending the prompt and what came before."""
    rng = torch.Generator().manual_seed(3)
    Hq, Hkv, D, BS, n, prompt, steps = 16, 4, 128, 16, 5, 200, 4
    shared = prompt // BS * BS  # the partial block is each request's own
    per = -(-(prompt + steps) // BS)
    nb = 2 + shared // BS + n * (per - shared // BS)
    rows = lambda *s: torch.randn(s, generator=rng).bfloat16()
    k_cache, v_cache = rows(nb, BS, Hkv, D).cuda(), rows(nb, BS, Hkv, D).cuda()
    perm = np.random.default_rng(1).permutation(np.arange(2, nb))
    table = np.zeros((n, per), np.int32)
    table[:, : shared // BS] = perm[: shared // BS]
    table[:, shared // BS:] = perm[shared // BS:].reshape(n, -1)
    slot = lambda r, p: table[r, p // BS].astype(np.int64) * BS + p % BS
    pk, pv = rows(prompt, Hkv, D), rows(prompt, Hkv, D)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    # the prompt: one prefill step of request 0, then the tail block's rows for the others
    qsl, seq = np.array([0, prompt], np.int32), np.array([prompt], np.int32)
    q0 = rows(prompt, Hq, D).cuda()
    cb.paged_attention(torch.empty_like(q0), q0, k_cache, v_cache, dev(qsl), dev(seq), dev(table[:1]), qsl, seq,
                       cb.alloc_workspace(1, prompt, Hq, Hkv, D), k_new=pk.cuda(), v_new=pv.cuda(),
                       slot_mapping=dev(slot(0, np.arange(prompt))))
    tail = np.arange(shared, prompt)
    for r in range(1, n):
        cb.write_kv(pk[shared:].cuda(), pv[shared:].cuda(), k_cache, v_cache, dev(slot(r, tail)))
    ws = cb.alloc_workspace_shared(n, n, Hq, Hkv, D)
    plen = np.full(n, shared, np.int32)
    group = np.array([0, n], np.int32)
    mine = [([pk], [pv]) for _ in range(n)]
    for i in range(steps):
        q, k, v = rows(n, Hq, D), rows(n, Hkv, D), rows(n, Hkv, D)
        qsl, seq = np.arange(n + 1, dtype=np.int32), np.full(n, prompt + i + 1, np.int32)
        out = torch.empty((n, Hq, D), dtype=torch.bfloat16, device="cuda")
        cb.paged_attention_shared(out, q.cuda(), k_cache, v_cache, dev(qsl), dev(seq), dev(table), dev(plen), qsl,
                                  seq, plen, group, ws, k_new=k.cuda(), v_new=v.cuda(),
                                  slot_mapping=dev(np.array([slot(r, np.int64(prompt + i)) for r in range(n)])),
                                  flags=cb.CB_FLAG_SHARE_ALWAYS)
        for r in range(n):
            mine[r][0].append(k[r:r + 1])
            mine[r][1].append(v[r:r + 1])
            K, V = (torch.cat(x).double().numpy() for x in mine[r])
            for g in range(Hkv):
                heads = slice(4 * g, 4 * g + 4)
                ref = oracle.paged_kv.softmax_attend(q[r, heads].double().numpy(), K[:, g], V[:, g], D ** -0.5)
                absv = oracle.paged_kv.softmax_attend(q[r, heads].double().numpy(), K[:, g], np.abs(V[:, g]), D ** -0.5)
                got = out[r, heads].double().cpu().numpy()
                # bf16 outputs and weights: 2^-8 of the value and of the mean |V|; scores 2^-15 B, B < 2^6 here
                assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -9) * absv).all()
    assert cb.read_error_word(ws) == 0
