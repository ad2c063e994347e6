"""The 8-bit paged cache on the GPU against the float64 oracle: writes bit for bit, reads exactly,
attention within bounds derived from the roundings of its arithmetic."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_attention_cb_gb300 as cb
import workloads
from oracle import kv_q8

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def launches(name):
    return cb.launch_count(cb.kernel_names().index(name))


def host_rows(rng, shape, dtype):
    """Rows whose size differs from row to row, as the values of `dtype` (exact in float64)."""
    x = rng.normal(size=shape) * np.exp(0.7 * rng.normal(size=shape[:-1]))[..., None]
    return torch.from_numpy(x).to(TORCH[dtype])


class Q8Step:
    """A StepSpec with an 8-bit pool (host codes and device tensors)."""

    def __init__(self, spec, seed=0, chunk=None):
        self.spec = s = spec
        rng = np.random.default_rng(seed)
        shape = (s.num_blocks, s.block_size, s.num_kv_heads, s.head_dim)
        pool = lambda: list(kv_q8.codes(*kv_q8.quantise_rows(host_rows(rng, shape, "f32").double().numpy())))
        self.k, self.v = pool(), pool()
        self.q = host_rows(rng, (s.T, s.num_q_heads, s.head_dim), s.dtype)
        self.k_new = host_rows(rng, (s.T, s.num_kv_heads, s.head_dim), s.dtype)
        self.v_new = host_rows(rng, (s.T, s.num_kv_heads, s.head_dim), s.dtype)
        self.md = workloads.metadata_tensors(s, "cuda")
        if chunk is None:
            chunk = int(s.seq_lens[s.q_lens > 1].sum())
        self.ws = cb.alloc_workspace_q8(s.R, s.T, s.num_q_heads, s.num_kv_heads, s.head_dim,
                                        s.block_size, chunk)
        self.upload()

    def upload(self):
        self.d = [cuda(self.k[0]), cuda(self.v[0]), cuda(self.k[1]), cuda(self.v[1])]
        self.dq, self.dk, self.dv = self.q.cuda(), self.k_new.cuda(), self.v_new.cuda()

    def run(self, flags=0, out=None, new=True, ws=None, stream=None):
        s = self.spec
        if out is None:
            out = torch.full_like(self.dq, float("nan"))
        kw = dict(k_new=self.dk, v_new=self.dv, slot_mapping=self.md["slot_mapping"]) if new else {}
        return cb.paged_attention_q8(out, self.dq, *self.d, self.md["query_start_loc"], self.md["seq_lens"],
                                     self.md["block_table"], s.query_start_loc, s.seq_lens,
                                     self.ws if ws is None else ws, scale=s.scale,
                                     sliding_window=s.sliding_window, flags=flags, stream=stream, **kw)

    def oracle(self, new=True):
        """(float64 output, bound): what the arithmetic's roundings add up to at most.

        With w the softmax weights, A = sum w |V| and B = max_j scale * sum |q| |K_j|:
        a score is a sum of up to 128 exact products in fp32, off by at most 2^-16 B in natural
        units (128 additions of 2^-23, the tensor cores truncate), which moves a weight by a
        factor 1 +- 2^-15 B; exponentials and scalings 2^-20; sums over n keys n 2^-23; fp16 weights
        2^-11 (bf16 queries), two fp16 parts 2^-21 (fp32 queries); bf16 weights on the prefill
        tiles 2^-8; the output's own rounding 2^-8 (bf16) or 2^-24 of its value.
        """
        s = self.spec
        k, v = [a.copy() for a in self.k], [a.copy() for a in self.v]
        if new:
            kv_q8.write_kv(*k, self.k_new.double().numpy(), s.slot_mapping)
            kv_q8.write_kv(*v, self.v_new.double().numpy(), s.slot_mapping)
        kc, vc = kv_q8.values(*k), kv_q8.values(*v)
        q = self.q.double().numpy()
        att = lambda a, b, c: oracle.paged_attention(a, b, c, s.query_start_loc, s.seq_lens, s.block_table,
                                                     s.block_size, s.scale, s.sliding_window)
        ref, absv = att(q, kc, vc), att(q, kc, np.abs(vc))
        G = s.num_q_heads // s.num_kv_heads
        B = np.zeros(q.shape[:2])
        for r in range(s.R):
            kk = oracle.paged_kv.gather_request_kv(np.abs(kc), s.block_table[r], int(s.seq_lens[r]), s.block_size)
            for t in range(s.query_start_loc[r], s.query_start_loc[r + 1]):
                for h in range(s.num_q_heads):
                    B[t, h] = s.scale * (kk[:, h // G] @ np.abs(q[t, h])).max()
        n = int(s.seq_lens.max())
        if s.dtype == "f32":
            rel, w = 2.0 ** -24, 2.0 ** -21
        else:
            chunk = np.repeat(s.q_lens > 1, s.q_lens)[:, None, None]
            rel, w = 2.0 ** -8, np.where(chunk, 2.0 ** -8, 2.0 ** -11)
        return ref, rel * np.abs(ref) + (2.0 ** -15 * B[..., None] + 2.0 ** -20 + n * 2.0 ** -23 + w) * absv

    def check(self, out, new=True):
        ref, tol = self.oracle(new)
        got = out.double().cpu().numpy()
        assert np.isfinite(got).all()
        bad = np.abs(got - ref) > tol
        assert not bad.any(), (int(bad.sum()), float((np.abs(got - ref) / tol).max()))

    def check_cache(self):
        k, v = [a.copy() for a in self.k], [a.copy() for a in self.v]
        kv_q8.write_kv(*k, self.k_new.double().numpy(), self.spec.slot_mapping)
        kv_q8.write_kv(*v, self.v_new.double().numpy(), self.spec.slot_mapping)
        for got, want in zip(self.d, (k[0], v[0], k[1], v[1])):
            assert np.array_equal(got.cpu().numpy(), want)


# ------------------------------------------------------------------ writing and reading


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,D,BS", [(1, 1, 64, 1), (1, 8, 128, 16), (7, 3, 64, 2), (33, 5, 128, 32),
                                      (200, 8, 128, 16), (129, 16, 64, 256)])
def test_write_then_read(T, H, D, BS, dtype):
    rng = np.random.default_rng(T * 7 + H)
    nb = 3 + -(-2 * T // BS)
    slots = rng.permutation(nb * BS)[:T].astype(np.int64)
    slots[::5] = -1
    x = [host_rows(rng, (T, H, D), dtype) for _ in range(2)]
    if T > 6:
        x[0][1] = 0.0
        x[0][2, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 1.0])
        x[0][3, 0] = torch.tensor(1e-38).to(x[0].dtype)   # scales at the lower end
        x[0][4, 0] = 3e38
        x[0][6, 0, 1] = 1e-30
        if dtype == "f32":
            x[0][6, 1, :] = 2.0 ** -149
    code = [rng.integers(0, 127, (nb, BS, H, D)).astype(np.uint8) for _ in range(2)]
    scale = [rng.integers(100, 140, (nb, BS, H)).astype(np.uint8) for _ in range(2)]
    d = [cuda(a).view(torch.float8_e4m3fn) for a in code] + [cuda(a).view(torch.float8_e8m0fnu) for a in scale]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cb.write_kv_q8(x[0].cuda(), x[1].cuda(), *d, cuda(slots), err)
    for i in range(2):
        kv_q8.write_kv(code[i], scale[i], x[i].double().numpy(), slots)
        assert np.array_equal(d[2 + i].view(torch.uint8).cpu().numpy(), scale[i])
        got, want = d[i].view(torch.uint8).cpu().numpy(), code[i]
        nan = (want & 0x7F) == 0x7F
        assert np.array_equal((got & 0x7F)[nan], want[nan] & 0x7F)
        assert np.array_equal(got[~nan], want[~nan])
    assert int(err) == 0
    # read back, in another order, a slot twice, two rows left as they were
    at = np.where(slots < 0, slots.max(), slots)[::-1].copy()
    at[: min(2, T - 1)] = -1
    for out_t in ("f32", "bf16"):
        o = [torch.full((T, H, D), 5.0, dtype=TORCH[out_t], device="cuda") for _ in range(2)]
        cb.read_kv_q8(*d, cuda(at), *o, err)
        for i in range(2):
            want = kv_q8.values(code[i], scale[i]).reshape(nb * BS, H, D)[np.maximum(at, 0)]
            want = torch.from_numpy(np.where((at < 0)[:, None, None], 5.0, want)).to(TORCH[out_t])
            assert torch.equal(o[i].cpu().nan_to_num(nan=-7.0), want.nan_to_num(nan=-7.0))
    assert int(err) == 0


def test_slots_past_the_pool_are_recorded_and_skipped():
    H, D, BS, nb = 2, 64, 16, 4
    d = [torch.zeros((nb, BS, H, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    d += [torch.zeros((nb, BS, H), dtype=torch.uint8, device="cuda") for _ in range(2)]
    x = torch.randn((3, H, D), device="cuda")
    for slots, want in (([0, 64, 5], 2), ([1, -3, 2 ** 40], 2), ([1, 2, 63], 0)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        s = torch.tensor(slots, device="cuda")
        cb.write_kv_q8(x, x, *d, s, err)
        assert int(err) == want
        err.zero_()
        o = torch.full_like(x, 9.0)
        cb.read_kv_q8(*d, s, o, torch.empty_like(o), err)
        assert int(err) == want
        for i, t in enumerate(slots):
            if not 0 <= t < nb * BS:
                assert (o[i] == 9.0).all()
            else:
                assert (o[i] - x[i]).abs().max() <= x[i].abs().max() * 2.0 ** -4


# ------------------------------------------------------------------ attention


def spec_of(q, ctx, **kw):
    kw.setdefault("pool_factor", 1.3)
    return workloads.custom(q, ctx, **kw)


DECODE = [
    dict(q=[1], ctx=[0]),
    dict(q=[1], ctx=[15]),
    dict(q=[1], ctx=[16]),
    dict(q=[1, 0, 1, 1], ctx=[300, 40, 0, 1000]),
    dict(q=[1] * 9, ctx=[0, 1, 14, 15, 16, 17, 31, 32, 700]),
    dict(q=[1] * 3, ctx=[5000, 3, 2000]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D,BS", [(32, 8, 128, 16), (8, 8, 64, 32), (16, 1, 128, 16), (4, 2, 64, 16),
                                         (64, 8, 128, 64), (10, 5, 128, 128), (12, 12, 64, 16), (16, 16, 128, 256)])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode(case, Hq, Hkv, D, BS, dtype):
    c = DECODE[case]
    st = Q8Step(spec_of(c["q"], c["ctx"], num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, block_size=BS,
                        dtype=dtype, seed=case), seed=case + 10)
    out = st.run()
    st.check(out)
    st.check_cache()
    assert cb.read_error_word(st.ws) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [1, 15, 16, 17, 100, 100000])
@pytest.mark.parametrize("Hq,Hkv,D,BS", [(32, 8, 128, 16), (4, 4, 64, 32)])
def test_window(Hq, Hkv, D, BS, W, dtype):
    st = Q8Step(spec_of([1, 3, 1, 6], [700, 40, 5, 130], num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D,
                        block_size=BS, dtype=dtype, sliding_window=W, seed=4), seed=W)
    st.check(st.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D,BS", [(32, 8, 128, 16), (8, 1, 64, 16), (16, 1, 128, 32), (4, 4, 64, 64)])
def test_query_runs(Hq, Hkv, D, BS, dtype):
    """Runs of query tokens around the tile sizes, decode rows between them."""
    st = Q8Step(spec_of([2, 1, 8, 9, 0, 33, 16, 1], [0, 77, 5, 300, 9, 64, 15, 0], num_q_heads=Hq,
                        num_kv_heads=Hkv, head_dim=D, block_size=BS, dtype=dtype, seed=1), seed=2)
    st.check(st.run())
    st.check_cache()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (8, 2, 64), (16, 1, 128)])
@pytest.mark.parametrize("columns", [16, 32, 64])
def test_runs_of_one_length(columns, Hq, Hkv, D, dtype):
    """Drafts of every request: items of each width."""
    n = columns * Hkv // Hq
    st = Q8Step(spec_of([n] * 5, [0, 31, 300, 1500, 90], num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D,
                        dtype=dtype, seed=1), seed=2)
    st.check(st.run())
    st.check_cache()


@pytest.mark.parametrize("dtype,W", [("bf16", 0), ("bf16", 150), ("f32", 0)])
@pytest.mark.parametrize("Hq,Hkv,D,BS", [(8, 2, 128, 16), (4, 4, 64, 128), (16, 1, 64, 256)])
def test_chunks_and_decodes(Hq, Hkv, D, BS, dtype, W):
    st = Q8Step(spec_of([1, 130, 1, 257, 70], [90, 0, 400, 333, 128], num_q_heads=Hq, num_kv_heads=Hkv,
                        head_dim=D, block_size=BS, dtype=dtype, sliding_window=W, seed=6), seed=3)
    st.check(st.run())
    st.check_cache()
    assert cb.read_error_word(st.ws) == 0


@pytest.mark.parametrize("W", [0, 600])
@pytest.mark.parametrize("Hq,Hkv,D,BS", [(32, 8, 128, 16), (16, 16, 128, 128), (32, 16, 64, 32), (16, 1, 64, 256),
                                         (32, 8, 128, 8)])
def test_long_chunks_and_decodes(Hq, Hkv, D, BS, W):
    """Runs that are computed from bf16 copies of their pages, between decode rows."""
    st = Q8Step(spec_of([1, 530, 1, 257, 170], [90, 0, 400, 1333, 2128], num_q_heads=Hq, num_kv_heads=Hkv,
                        head_dim=D, block_size=BS, sliding_window=W, seed=6), seed=3)
    before = launches("dequant_pages")
    st.check(st.run())
    st.check_cache()
    assert launches("dequant_pages") == before + 1
    assert cb.read_error_word(st.ws) == 0


def test_more_chunks_than_one_launch_lists():
    st = Q8Step(spec_of([70, 90] * 65, [60, 100] * 65, num_q_heads=8, num_kv_heads=2, head_dim=64, seed=1), seed=1)
    before = launches("dequant_pages")
    st.check(st.run())
    st.check_cache()
    assert launches("dequant_pages") == before + 2


@pytest.mark.parametrize("Hq,Hkv,D,BS,W,q,ctx", [
    (8, 2, 128, 16, 0, [200], [15000]),            # three pairs of query tiles and a tail
    (4, 4, 64, 128, 0, [129, 1, 70], [12900, 800, 16001]),
    (16, 1, 64, 32, 0, [30, 5], [37000, 42000]),   # two full tiles; a tail of five tokens
    (8, 2, 128, 16, 5500, [257], [9000]),
    (8, 2, 128, 256, 0, [512, 65], [3000, 14000]),  # pairs of one and of many units
])
def test_few_chunks_behind_long_contexts(Hq, Hkv, D, BS, W, q, ctx):
    """The keys of too few query tiles to fill the GPU are split; the pieces are merged."""
    st = Q8Step(spec_of(q, ctx, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, block_size=BS,
                        sliding_window=W, seed=6), seed=3)
    before = launches("merge_rows"), launches("dequant_pages")
    st.check(st.run())
    st.check_cache()
    assert launches("merge_rows") > before[0] and launches("dequant_pages") == before[1] + 1
    assert cb.read_error_word(st.ws) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D,BS", [(8, 2, 128, 1), (4, 4, 64, 4), (16, 1, 64, 8), (16, 1, 64, 2)])
def test_small_pages_run_on_the_portable_kernel(Hq, Hkv, D, BS, dtype):
    before = cb.launch_count(cb.kernel_names().index("portable_q8"))
    st = Q8Step(spec_of([1, 5, 0, 1], [40, 3, 2, 0], num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D,
                        block_size=BS, dtype=dtype, sliding_window=20, seed=8), seed=5)
    st.check(st.run())
    st.check_cache()
    assert cb.launch_count(cb.kernel_names().index("portable_q8")) == before + 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [0, 21])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 64), (32, 16, 64), (20, 10, 128), (32, 8, 128)])
def test_pages_of_eight(Hq, Hkv, D, W, dtype):
    """Key blocks of two pages: ends in the first and the second, new rows in either, values of
    unattended slots, and a chunk."""
    spec = spec_of([1, 5, 1, 1, 0, 1, 40, 1], [0, 3, 7, 8, 2, 23, 300, 1001], num_q_heads=Hq, num_kv_heads=Hkv,
                   head_dim=D, block_size=8, dtype=dtype, sliding_window=W, seed=8)
    st = Q8Step(spec, seed=5)
    before = launches("portable_q8")
    out = st.run()
    st.check(out)
    st.check_cache()
    used = np.zeros(spec.num_blocks * 8, bool)
    for r in range(spec.R):
        first = max(0, int(spec.ctx_lens[r]) - W + 1) if W else 0
        for p in range(first, int(spec.seq_lens[r])):
            used[spec.block_table[r, p // 8] * 8 + p % 8] = True
    keep = torch.from_numpy(used).cuda().view(spec.num_blocks, 8)
    for i in range(4):
        st.d[i][~keep] = 0x7F if i < 2 else 0xFF
    assert torch.equal(st.run(), out)
    assert cb.read_error_word(st.ws) == 0
    assert launches("portable_q8") == before


@pytest.mark.parametrize("q", [1, 3])
def test_decode_rows_in_pages_of_eight(q):
    """Decode rows alone (the new rows are written by the kernel that reads them), or runs."""
    st = Q8Step(spec_of([q] * 9, [0, 1, 6, 7, 8, 15, 16, 700, 3001], block_size=8, seed=3), seed=4)
    before = launches("portable_q8")
    st.check(st.run())
    st.check_cache()
    assert launches("portable_q8") == before


def test_a_bad_second_page_of_eight_reads_as_zeros():
    spec = spec_of([1, 1], [100, 60], block_size=8, seed=2)
    spec.block_table[0, 3] = spec.num_blocks + 5
    spec.block_table[1, 5] = -1
    st = Q8Step(spec, seed=1)
    out = st.run()
    assert cb.read_error_word(st.ws) == cb.CB_DEVERR_BLOCK_ID
    for a in (st.k, st.v):
        a[0] = np.concatenate([a[0], np.zeros_like(a[0][:1])])
        a[1] = np.concatenate([a[1], np.full_like(a[1][:1], 127)])
    spec.block_table[0, 3] = spec.block_table[1, 5] = spec.num_blocks
    st.check(out)


def test_portable_flag_agrees():
    st = Q8Step(spec_of([1, 4, 1], [50, 20, 333], seed=2), seed=1)
    st.check(st.run(flags=cb.CB_FLAG_PORTABLE_ONLY))


def test_without_new_rows():
    st = Q8Step(spec_of([1, 2], [50, 20], seed=2), seed=1)
    st.check(st.run(new=False), new=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q", [[1, 1], [5, 1]])
def test_values_of_unattended_slots_do_not_matter(q, dtype):
    """NaN codes and any scale in slots behind the sequences, in front of the window and in
    pages of nobody leave the output as it is."""
    spec = spec_of(q, [100, 37], dtype=dtype, sliding_window=30, seed=2)
    st = Q8Step(spec, seed=1)
    clean = st.run().clone()
    used = np.zeros(spec.num_blocks * spec.block_size, bool)
    for r in range(spec.R):
        for p in range(max(0, int(spec.ctx_lens[r]) - 30 + 1), int(spec.seq_lens[r])):
            used[spec.block_table[r, p // spec.block_size] * spec.block_size + p % spec.block_size] = True
    keep = torch.from_numpy(used).cuda().view(spec.num_blocks, spec.block_size)
    for i in range(4):
        st.d[i][~keep] = 0x7F if i < 2 else 0xFF
    assert torch.equal(st.run(), clean)


@pytest.mark.parametrize("ctx", [500, 15000])
@pytest.mark.parametrize("W,BS", [(0, 16), (30, 16), (60, 16), (150, 128)])
def test_values_of_unattended_slots_do_not_matter_to_chunks(W, BS, ctx):
    spec = spec_of([2000, 70], [ctx, 37], sliding_window=W, block_size=BS, seed=2)
    st = Q8Step(spec, seed=1)
    before = launches("dequant_pages")
    clean = st.run().clone()
    assert launches("dequant_pages") == before + (W != 30)  # (a small window: little work)
    used = np.zeros(spec.num_blocks * BS, bool)
    for r in range(spec.R):
        first = max(0, int(spec.ctx_lens[r]) - W + 1) if W else 0
        for p in range(first, int(spec.seq_lens[r])):
            used[spec.block_table[r, p // BS] * BS + p % BS] = True
    keep = torch.from_numpy(used).cuda().view(spec.num_blocks, BS)
    for i in range(4):
        st.d[i][~keep] = 0x7F if i < 2 else 0xFF
    assert torch.equal(st.run(), clean)


def shifted(t):
    """The same tensor 16 bytes behind an address that is a multiple of 256."""
    flat = torch.empty(t.numel() + 16 // t.element_size(), dtype=t.dtype, device=t.device)
    return flat[16 // t.element_size():].view(t.shape).copy_(t)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q,ctx", [([1, 1, 1], [700, 20, 3000]), ([1, 200, 3], [700, 4000, 50])])
def test_addresses_aligned_to_sixteen_bytes(q, ctx, dtype):
    st = Q8Step(spec_of(q, ctx, dtype=dtype, seed=4), seed=4)
    st.d = [shifted(t) for t in st.d]
    st.dq, st.dk, st.dv, st.ws = (shifted(t) for t in (st.dq, st.dk, st.dv, st.ws))
    st.check(st.run(out=shifted(torch.full_like(st.dq, float("nan")))))
    st.check_cache()
    k, v = torch.empty_like(st.dk), torch.empty_like(st.dv)
    cb.read_kv_q8(*st.d, st.md["slot_mapping"], shifted(k), shifted(v))


@pytest.mark.parametrize("Hkv,portable", [(7, False), (11, False), (128, False), (129, True)])
def test_any_number_of_heads(Hkv, portable):
    """Heads that a CTA's eight do not divide, the most the tensor-core kernel takes, and more."""
    i = cb.kernel_names().index("portable_q8")
    before = cb.launch_count(i)
    st = Q8Step(spec_of([1, 4, 70], [90, 33, 40], num_q_heads=Hkv, num_kv_heads=Hkv, head_dim=64, seed=4), seed=4)
    st.check(st.run())
    assert cb.launch_count(i) == before + portable


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_very_different_scale(dtype):
    """K rows from 2^-20 to 2^6 and V rows from 2^-60 to 2^60 in one context: the weights of the
    attended keys keep their precision whatever the scales of the others."""
    spec = spec_of([1, 3], [200, 60], dtype=dtype, seed=2)
    st = Q8Step(spec, seed=1)
    rng = np.random.default_rng(5)
    st.k[1][:] = rng.integers(107, 121, st.k[1].shape)
    st.v[1][:] = rng.integers(67, 187, st.v[1].shape)
    st.upload()
    st.check(st.run())


def test_queries_of_extreme_size():
    spec = spec_of([1, 2], [100, 30], dtype="f32", seed=2)
    st = Q8Step(spec, seed=1)
    st.q[0] *= 2.0 ** -100
    st.q[1, 1:] = 0.0
    st.q[2, 0, 0] *= 2.0 ** 12
    st.upload()
    st.check(st.run())


def test_bad_page_ids_read_as_zeros():
    spec = spec_of([1, 1], [100, 60], seed=2)
    spec.block_table[0, 2] = spec.num_blocks + 5
    spec.block_table[1, 1] = -1
    st = Q8Step(spec, seed=1)
    out = st.run()
    assert torch.isfinite(out.float()).all()
    assert cb.read_error_word(st.ws) == cb.CB_DEVERR_BLOCK_ID
    # the pages' keys score zero and their values are zero
    nb = spec.num_blocks
    for a in (st.k, st.v):
        a[0] = np.concatenate([a[0], np.zeros_like(a[0][:1])])
        a[1] = np.concatenate([a[1], np.full_like(a[1][:1], 127)])
    spec.block_table[0, 2] = spec.block_table[1, 1] = nb
    st.check(out)


def test_steps_of_any_size_share_a_workspace():
    ws = cb.alloc_workspace_q8(64, 600, 32, 8, 128, 16, 6000)
    for q, ctx in (([1] * 40, list(range(0, 1200, 30))), ([1], [3000]), ([300, 1, 4], [5000, 800, 20]), ([300, 1, 4], [500, 800, 20]), ([1] * 3, [9, 90, 900])):
        st = Q8Step(spec_of(q, ctx, seed=len(q)), seed=len(q))
        st.check(st.run(ws=ws))
    assert cb.read_error_word(ws) == 0


def test_many_requests_and_many_pieces():
    """More rows to merge than one launch lists, and one request over every SM."""
    st = Q8Step(spec_of([1] * 300, [16 * (i % 3) + 70 for i in range(300)], num_q_heads=8, num_kv_heads=2,
                        head_dim=64, seed=1), seed=1)
    st.check(st.run())
    st = Q8Step(spec_of([1], [20000], num_q_heads=8, num_kv_heads=2, head_dim=64, seed=1), seed=2)
    st.check(st.run())


@pytest.mark.parametrize("q,ctx", [([1, 3, 100], [700, 50, 20]), ([1, 3, 200], [700, 50, 6000])])
def test_graph_replay_and_side_stream(q, ctx):
    st = Q8Step(spec_of(q, ctx, seed=3), seed=3)
    s = torch.cuda.Stream()
    out = torch.full_like(st.dq, float("nan"))
    with torch.cuda.stream(s):
        st.run(out=out)
        st.run(out=out)
    s.synchronize()
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.run(out=out)
    for i in range(3):
        out.fill_(float("nan"))
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # new values in the same buffers
    st.q = host_rows(np.random.default_rng(9), tuple(st.q.shape), "bf16")
    st.dq.copy_(st.q)
    g.replay()
    torch.cuda.synchronize()
    st.check(out)


def test_decoding_in_sequence():
    """A prompt is written in a chunk and tokens follow one by one, each attending what the steps
    before it stored; the rows read back at the end are the ones written."""
    H, D, BS, nb = 2, 128, 16, 12
    rng = np.random.default_rng(0)
    d = [torch.randint(0, 256, (nb, BS, H, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    d += [torch.randint(1, 255, (nb, BS, H), dtype=torch.uint8, device="cuda") for _ in range(2)]
    table = rng.permutation(nb)[:8].astype(np.int32)
    ws = cb.alloc_workspace_q8(1, 90, 8, H, D, BS, 100)
    all_k = host_rows(rng, (100, H, D), "bf16")
    all_v = host_rows(rng, (100, H, D), "bf16")
    slots = table[np.arange(100) // BS].astype(np.int64) * BS + np.arange(100) % BS
    vk, vv = (lambda x: (lambda y, e: y * np.exp2(e.astype(float))[..., None])(*kv_q8.quantise_rows(x.double().numpy())))(all_k), None
    vv = (lambda y, e: y * np.exp2(e.astype(float))[..., None])(*kv_q8.quantise_rows(all_v.double().numpy()))
    pos = 0
    for n in (90, 1, 1, 3, 1, 1, 1, 2):
        q = host_rows(rng, (n, 8, D), "bf16")
        qsl, seq = np.array([0, n], np.int32), np.array([pos + n], np.int32)
        out = torch.empty((n, 8, D), dtype=torch.bfloat16, device="cuda")
        cb.paged_attention_q8(out, q.cuda(), *d, cuda(qsl), cuda(seq), cuda(table[None]), qsl, seq, ws,
                              k_new=all_k[pos:pos + n].cuda(), v_new=all_v[pos:pos + n].cuda(),
                              slot_mapping=cuda(slots[pos:pos + n]))
        cache = lambda v: v[:pos + n].reshape(1, pos + n, H, D)
        ref = oracle.paged_attention(q.double().numpy(), cache(vk), cache(vv), qsl, seq, np.zeros((1, 1), np.int32),
                                     pos + n, 1.0 / np.sqrt(D))
        # bf16 outputs 2^-8 of the value, bf16 or fp16 weights 2^-8 of the largest V
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * np.abs(vv[:pos + n]).max()
        assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
        pos += n
    o = [torch.empty((100, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cb.read_kv_q8(*d, cuda(slots), *o)
    assert np.array_equal(o[0].double().cpu().numpy(), vk) and np.array_equal(o[1].double().cpu().numpy(), vv)
    assert cb.read_error_word(ws) == 0


def test_two_streams_with_their_own_workspaces():
    a = Q8Step(spec_of([1] * 8, [500 + 90 * i for i in range(8)], seed=1), seed=1)
    b = Q8Step(spec_of([1] * 5, [900 + 190 * i for i in range(5)], seed=2), seed=2)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(5):
        with torch.cuda.stream(sa):
            oa = a.run()
        with torch.cuda.stream(sb):
            ob = b.run()
        outs.append((oa, ob))
    torch.cuda.synchronize()
    for oa, ob in outs:
        assert torch.equal(oa, outs[0][0]) and torch.equal(ob, outs[0][1])
    a.check(outs[0][0])
    b.check(outs[0][1])


def test_binding_refuses():
    st = Q8Step(spec_of([1], [20], seed=1), seed=1)
    args = (st.md["query_start_loc"], st.md["seq_lens"], st.md["block_table"], st.spec.query_start_loc,
            st.spec.seq_lens, st.ws)
    out = torch.empty_like(st.dq)
    for bad in (out.float(), out[:, :4], out.transpose(0, 1), out.cpu()):
        with pytest.raises(cb.CbError):
            cb.paged_attention_q8(bad, st.dq, *st.d, *args)
    for i in range(4):
        d = list(st.d)
        d[i] = d[i][:, :8] if i < 2 else d[i].float()
        with pytest.raises(cb.CbError):
            cb.paged_attention_q8(out, st.dq, *d, *args)
    with pytest.raises(cb.CbError):
        cb.paged_attention_q8(out, st.dq, *st.d, *args, k_new=st.dk)
    with pytest.raises(cb.CbError):
        cb.write_kv_q8(st.dk, st.dv, *st.d, st.md["slot_mapping"].int())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_a_nan_reaches_only_the_rows_that_attend_it(D, dtype):
    """A NaN in one token's V row: the earlier tokens of the same run stay finite, the ones that
    attend it are NaN in that element and nowhere else."""
    for n, W in ((2, 0), (5, 0), (5, 3), (13, 0)):
        spec = spec_of([n, 1], [21, 60], num_q_heads=4, num_kv_heads=2, head_dim=D, dtype=dtype, sliding_window=W, seed=n)
        st = Q8Step(spec, seed=n)
        clean = st.run().clone()
        st.v_new[n // 2, 1, 37] = float("nan")
        st.upload()
        got = st.run()
        pos = np.arange(n)
        hit = torch.from_numpy((pos >= n // 2) & ((W == 0) | (pos - n // 2 < W)))
        want = torch.zeros(got.shape, dtype=torch.bool)
        want[:n, 2:, 37] = hit[:, None]
        assert torch.equal(torch.isnan(got).cpu(), want)
        assert torch.equal(got[~want.cuda()], clean[~want.cuda()])


def test_new_rows_go_where_their_slots_say():
    """Decode rows with a slot of -1, one in a page of nobody and one past the pool: the cache and
    the attended values are those of a write before the attention."""
    spec = spec_of([1, 1, 1, 1], [40, 21, 100, 3], seed=3)
    spec.slot_mapping[1] = -1
    spare = sorted(set(range(2, spec.num_blocks)) - set(spec.block_table.reshape(-1).tolist()))
    spec.slot_mapping[2] = spare[0] * 16 + 5
    st = Q8Step(spec, seed=3)
    st.check(st.run())
    st.check_cache()
    assert cb.read_error_word(st.ws) == 0
    spec.slot_mapping[3] = spec.num_blocks * 16
    st = Q8Step(spec, seed=3)
    out = st.run()
    assert cb.read_error_word(st.ws) == cb.CB_DEVERR_SLOT
    spec.slot_mapping[3] = -1  # skipped: as if it had none
    st.check(out)
    st.check_cache()
