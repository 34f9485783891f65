"""Latent attention where its calls can go wrong, on the GPU against the float64 definitions of latent_ref."""
import numpy as np
import pytest
import torch

from rotation_quantized_kv_rq_gb300 import rq
from tests import block_ref as R
from tests import latent_ref as L
from tests.test_latent_gpu import DT, Case, check_prompt, dev, gen, host, int32, make, prompt_case, within

pytestmark = pytest.mark.gpu

# a weight's pieces in the absorbed form, rounded to fp16 before
PIECES = {torch.bfloat16: 2.0 ** -8 + 2.0 ** -11, torch.float16: 2.0 ** -12 + 2.0 ** -11}


# --------------------------------------------------------------------------- the absorbed form

@pytest.mark.parametrize("heads", [9, 30, 70])
@pytest.mark.parametrize("power", [-120, 98, 107, 109, 118, 127])
def test_bf16_queries_of_any_magnitude(power, heads):
    """Queries of some 2^power against a scale of 2^-power.  Both are exact, so the definition is that of ordinary queries and a
    scale of 1; and the kernel splits a row by its own power of two, so its error is too."""
    case = Case(power & 7, [300, 20], 2, heads, 16, torch.bfloat16, sm_scale=2.0 ** -power, gain=0.07 * 2.0 ** power)
    if power == 127:
        case.q_c[0, 1, 0, 5] = torch.finfo(torch.bfloat16).max
    out = case.run()
    ref, tol = L.attention(host(case.q_c) * 2.0 ** -power, host(case.q_pe) * 2.0 ** -power, case.pages, case.table, case.lens, case.P,
                           L.chain(2), 1.0, torch.bfloat16)
    within(host(out), ref, tol + R.half_step(torch.bfloat16, ref) * (1 + 2.0 ** -8))


@pytest.mark.parametrize("heads", [9, 30, 70])
@pytest.mark.parametrize("power", [40, 90, 125])
def test_large_queries_across_large_latents(power, heads):
    """Query and latents of the largest magnitudes whose products are all zero: the mean of the latents.  The scales of the two
    multiply past float32's range."""
    rng, n, P, dtype = gen(power), 300, 16, torch.bfloat16
    c = rng.standard_normal((n, 512)) * 2.0 ** 66
    c[:, 0] = 0.0
    pages = np.zeros((n // P + 1, 641 * P), np.uint8)
    L.put(pages, P, np.arange(n), c, np.zeros((n, 64)), dtype)
    codes, _, byte = L.unpack(pages, P, dtype)
    c = (codes * L.scale(byte)[:, None])[:n]
    assert byte[:n].max() == 127 + 60
    cache = make(heads, P, len(pages), dtype, batch=1, sm_scale=1.0)
    cache.pages.copy_(torch.from_numpy(pages))
    q_c = torch.zeros(1, heads, 512, dtype=dtype, device="cuda")
    q_c[..., 0] = 2.0 ** power
    out = host(cache.decode(q_c, q_c.new_zeros(1, heads, 64), int32(np.arange(len(pages)))[None], int32([n])))
    ref = np.broadcast_to(c.mean(0), out.shape)
    tol = (PIECES[dtype] + 2.0 ** -20) * np.abs(c).mean(0)
    within(out, ref, tol + R.half_step(dtype, ref) * (1 + 2.0 ** -8))


@pytest.mark.parametrize("heads", [9, 30, 70])
def test_queries_times_scale_past_float32(heads):
    """A row whose largest value times sm_scale is past float32 is NaN; the others are as they were."""
    case = Case(2, [300, 20], 2, heads, 16, torch.bfloat16, sm_scale=2.0 ** 20, gain=0.07 * 2.0 ** -20)
    clean = case.run()
    case.q_c[0, 1, 3] = 2.0 ** 125
    case.q_pe[1, 0, 2] = -2.0 ** 127
    out = case.run()
    hit = torch.zeros(2, 2, heads, dtype=torch.bool, device="cuda")
    hit[0, 1, 3] = hit[1, 0, 2] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], clean[~hit]) and torch.isfinite(clean).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [3, 25, 70])
@pytest.mark.parametrize("power", [20, 24, 25, 26, 27, 28, 29, 33])
def test_attention_scores_of_any_magnitude(dtype, heads, power):
    """Scores up to 2^power and (in units of the exponential's) past it, whose largest rises through the tiles: the token with
    the largest has all the weight, however coarse float32's steps are there."""
    rng, n, P, dtype = gen(power), 600, 16, DT[dtype]
    c = rng.integers(-7, 8, (n, 512)) / 8.0
    c[:, 0], c[:, 1] = 0.25, 1.0
    c[5, 0], c[300, 0], c[599, 0] = 0.5, 0.75, 1.0
    pages = np.zeros((n // P + 1, 641 * P), np.uint8)
    L.put(pages, P, np.arange(n), c, np.zeros((n, 64)), dtype)
    cache = make(heads, P, len(pages), dtype, batch=1, sm_scale=2.0 ** power)
    cache.pages.copy_(torch.from_numpy(pages))
    q_c = torch.zeros(1, heads, 512, dtype=dtype, device="cuda")
    q_c[..., 0] = 1.0
    table = int32(np.arange(len(pages)))[None]
    for length, top in ((600, 599), (599, 300), (300, 5)):
        out = host(cache.decode(q_c, q_c.new_zeros(1, heads, 64), table, int32([length])))
        ref = np.broadcast_to(c[top], out.shape)
        within(out, ref, (PIECES[dtype] + 2.0 ** -20) * np.abs(ref) + R.half_step(dtype, ref), f"{length} tokens")


# ---------------------------------------------------------------------------- the expanded form

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("power", [-4, -1, 0, 1, 2, 3, 4, 8, 12])
def test_prompt_scores_of_any_magnitude(dtype, power):
    """Queries and keys of some 2,000, each query the same as its own key: that key's value is the result, however coarse float32's
    steps are at scores of 2^25 to 2^41."""
    rng, new, old, heads, dtype = gen(power + 20), 200, 300, 2, DT[dtype]
    q = dev(2000 * rng.standard_normal((new, heads, 192)), dtype)
    k = dev(2000 * rng.standard_normal((old + new, heads, 128)), dtype)
    k[old:] = q[..., :128]
    v = dev(rng.standard_normal((old + new, heads, 128)), dtype)
    out = rq.prompt_attention(q, k, k.new_zeros(old + new, 64), v, int32([0, new]), int32([0, old + new]), new, sm_scale=2.0 ** power)
    ref = host(v[old:])  # (the exponential is off by 2^-20 at most)
    within(host(out), ref, 2.0 ** -20 * np.abs(ref) + R.half_step(dtype, ref))


# ------------------------------------------------------------------------------------ streams

def beside(call, nbytes):
    """call(stream) while the current stream has yet to read memory of nbytes that is free again on the host's side: what the call
    allocates for itself is not that memory."""
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = call(s)
    torch.cuda.synchronize()
    want = [t.clone() for t in (want if isinstance(want, tuple) else (want,))]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    taken, kept = torch.full((nbytes,), 5, dtype=torch.uint8, device="cuda"), torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)  # some 0.2 s
    kept.copy_(taken)
    del taken
    got = call(s)
    s.synchronize()
    torch.cuda.synchronize()
    assert (kept == 5).all()
    for a, b in zip(got if isinstance(got, tuple) else (got,), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("raw", [False, True])
def test_stream_argument_of_the_prompt(raw):
    """The call's own workspace and output are not memory that the current stream still uses.  (Cut, so that it has parts.)"""
    q, k, pe, v, qo, ko = prompt_case(3, [64, 2], [5000, 3000], 2, torch.bfloat16)
    qo, ko = int32(qo), int32(ko)
    run = lambda s: rq.prompt_attention(q, k, pe, v, qo, ko, 64, stream=s.cuda_stream if raw else s)  # noqa: E731
    beside(run, rq.rq_prompt_workspace(0))
    out = run(torch.cuda.Stream())
    with torch.cuda.stream(torch.cuda.Stream()):
        zero = rq.prompt_attention(q, k, pe, v, qo, ko, 64, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(zero, out)
    check_prompt(out, q, k, pe, v, qo.tolist(), ko.tolist(), torch.bfloat16)


def test_stream_argument_of_the_cache():
    case = Case(5, [400, 70, 33, 9], 1, 128, 16, torch.float16)
    cache, tab, lens = case.cache, dev(case.table), dev(case.lens)
    q_c, q_pe = case.q_c[:, 0].contiguous(), case.q_pe[:, 0].contiguous()
    beside(lambda s: cache.decode(q_c, q_pe, tab, lens, stream=s), q_c.numel() * 2)
    beside(lambda s: cache.read(tab, int32([0, 400, 470, 503, 512]), 512, stream=s), 512 * 1024)
    n, rope = 200, rq.Rope(64)
    x, q = dev(gen(1).standard_normal((n, 576)), torch.float16), dev(gen(2).standard_normal((n, 128, 64)), torch.float16)
    slots, pos = torch.full((n,), -1, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")
    beside(lambda s: cache.append(x[:, :512], x[:, 512:], slots, rope, pos, q_pe=q, stream=s), n * 128 * 128)


def test_stream_argument_while_captured():
    """On the capturing stream and on one forked from it."""
    q, k, pe, v, qo, ko = prompt_case(3, [64, 2], [5000, 3000], 2, torch.bfloat16)
    qo, ko = int32(qo), int32(ko)
    case = Case(5, [400, 70, 33, 9], 1, 20, 16, torch.float16)
    q_c, q_pe, tab, lens = case.q_c[:, 0].contiguous(), case.q_pe[:, 0].contiguous(), dev(case.table), dev(case.lens)
    run = lambda s: (rq.prompt_attention(q, k, pe, v, qo, ko, 64, stream=s), case.cache.decode(q_c, q_pe, tab, lens, stream=s))  # noqa: E731
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    run(torch.cuda.current_stream())
    with torch.cuda.graph(graph):
        current = torch.cuda.current_stream()
        first = run(current)
        side.wait_stream(current)
        second = run(side)
        current.wait_stream(side)
    for t in (q, v, q_c):
        t.copy_(torch.randn_like(t))
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, run(None)):
        assert torch.equal(a, c) and torch.equal(b, c)


# ---------------------------------------------------------------------------------- refusals

def test_append_refuses_outputs_over_themselves():
    """Turned queries two of whose rows share elements; rows of tokens and heads that interleave do not."""
    n, heads, cache = 6, 4, make(4, 16, 4, torch.float16)
    x, buf = torch.zeros(n, 576, dtype=torch.float16, device="cuda"), torch.zeros(1 << 14, dtype=torch.float16, device="cuda")
    q, slots = dev(gen(1).standard_normal((n, heads, 64)), torch.float16), int32(range(n))
    call = lambda o, q=q: cache.append(x[:len(q), :512], x[:len(q), 512:], slots[:len(q)], q_pe=q, q_pe_out=o)  # noqa: E731
    for strides in ((256, 64), (64, 384), (64 * 3, 64 * 20), (128 * 4, 128), (64, 64 * 7), (72, 440), (256, 1728), (192, 448), (320, 128)):
        out = call(buf.as_strided((n, heads, 64), (*strides, 1)))
        assert torch.equal(out, q), strides
    for strides in ((64, 64), (128, 64), (192, 64), (64, 128), (64, 320), (248, 64), (72, 360), (256, 1024), (192, 128), (200, 64)):
        for in_place in (False, True):
            out = buf.as_strided((n, heads, 64), (*strides, 1))
            with pytest.raises(rq.RQError) as e:
                call(out, out if in_place else q)
            assert e.value.code == rq.RQ_ERR_INVALID, strides
    one = buf.as_strided((1, heads, 64), (8, 64, 1))  # a stride that is not used may be anything
    assert torch.equal(call(one, q[:1]), q[:1])


# ------------------------------------------------------------------- what other tests pass by

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [5, 20, 40])
def test_queries_with_an_outlier(dtype, heads):
    """One dim a thousand times the others: the pieces of a row have one scale, so the others' low bits are lost as
    latent_ref.attention counts them, and no more."""
    case = Case(heads, [500, 33], 2, heads, 32, DT[dtype], sm_scale=0.0024)
    case.q_c[..., 17] *= 1000
    case.q_c[:, :, 1, 300] *= -1000
    case.check(case.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_verify_of_many_rows_over_long_sequences(dtype):
    case = Case(7, [9000, 4100, 4], 4, 32, 64, DT[dtype])
    case.check(case.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new,old", [([3000] + [16] * 7, [0] * 8), ([64] * 20, [0] * 13 + [8000] + [5] * 6), ([1, 1500, 2], [2500, 10, 0])])
def test_prompts_of_very_different_lengths(dtype, new, old):
    dtype = DT[dtype]
    q, k, pe, v, qo, ko = prompt_case(len(new), new, old, 2, dtype)
    out = rq.prompt_attention(q, k, pe, v, int32(qo), int32(ko), max(new))
    check_prompt(out, q, k, pe, v, qo, ko, dtype)
    assert torch.equal(out, rq.prompt_attention(q, k, pe, v, int32(qo), int32(ko), max(new)))


@pytest.mark.parametrize("n,heads", [(300, 3), (200, 70), (1100, 2)])
def test_prompt_weights_of_nothing_and_all(n, heads):
    """Keys that are all the same, and scores that fall by 2^10 a key: means, and the row's own first keys."""
    rng, dtype = gen(n), torch.bfloat16
    q = torch.ones(n, heads, 192, dtype=dtype, device="cuda")
    k, pe = torch.ones(n, heads, 128, dtype=dtype, device="cuda"), torch.zeros(n, 64, dtype=dtype, device="cuda")
    v = dev(rng.standard_normal((n, heads, 128)), dtype)
    off = int32([0, n])
    check_prompt(rq.prompt_attention(q, k, pe, v, off, off, n), q, k, pe, v, [0, n], [0, n], dtype)
    pe[:, 0] = -1024.0 * torch.arange(n, device="cuda")
    out = host(rq.prompt_attention(q, k, pe, v, off, off, n, sm_scale=1.0))
    within(out, np.broadcast_to(host(v)[:1], out.shape), (2.0 ** -8 + 2.0 ** -20) * np.abs(host(v)[:1]))
