"""Rotary positions and the rotating append on the GPU against the double-precision
oracle: layouts, types, strides, directions, scalings, positions far out, the pages'
untouched parts, refusals at the Python front end, streams and captured graphs.

Tolerance of a rotated element, from the arithmetic: the angle is exact to 2^-26
half turns (pi 2^-26 < 2^-24 rad), sincospif is within 2 ulp (2^-23 at values up to
1), the magnitude, the two products and their sum round by 2^-24 each of at most
m (|x| + |y|); together below 2^-21 m (|x| + |y|).  The store rounds by half a step
of the type, eps / 2 relative (2^-25 absolute among fp16's subnormals).
"""
import numpy as np
import pytest
import torch

import oracle
from paged_latent_attention_gb300 import api, inputs

pytestmark = pytest.mark.gpu

PT, ROW = inputs.PAGE_TOKENS, inputs.ROW_ELEMS
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _bound(x, ref, layout, magnitude, dtype):
    a = np.abs(x)
    if layout == "half":
        s = a[..., : a.shape[-1] // 2] + a[..., a.shape[-1] // 2:]
        s = np.concatenate([s, s], axis=-1)
    else:
        s = np.repeat(a[..., 0::2] + a[..., 1::2], 2, axis=-1)
    fp32 = 2.0 ** -21 * abs(magnitude) * s
    return fp32 + torch.finfo(dtype).eps / 2 * (np.abs(ref) + fp32) + \
        (2.0 ** -25 if dtype == torch.float16 else 0.0)


def _f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H,dim,head,offset", [
    (1, 1, 64, 64, 0), (3, 16, 64, 192, 128), (5, 7, 128, 128, 0), (2, 3, 20, 27, 7),
    (700, 5, 32, 40, 8), (4, 128, 64, 64, 0), (2, 300, 2, 2, 0), (9, 2, 512, 512, 0)])
def test_rotation_matches_the_oracle(layout, kind, T, H, dim, head, offset):
    g = torch.Generator().manual_seed(T * 31 + H)
    full = torch.randn(T, H, head, generator=g).to(TYPES[kind]).cuda()
    x = full[..., offset:offset + dim]
    pos = torch.randint(-2**31, 2**31 - 1, (T,), generator=g, dtype=torch.int64).to(torch.int32)
    pos[0] = 0
    table = api.rope_table(dim, base=50000.0)
    freqs = oracle.rope_frequencies(dim, 50000.0)
    for inverse in (False, True):
        out = api.mla_rope(x, pos.cuda(), table, layout=layout, inverse=inverse)
        # positions up to 2^31 with frequencies in double: the oracle's own angle is
        # off by up to 2^31 * 2^-52 rad
        ref = oracle.rope_rotate(_f64(x), pos.numpy(), freqs, layout, 1.0, inverse)
        tol = _bound(_f64(x), ref, layout, 1.0, TYPES[kind]) + 2.0 ** -20 * np.abs(_f64(x)).max()
        assert np.all(np.abs(_f64(out) - ref) <= tol)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("scaling,kw", [
    ("linear", dict(factor=8.0)),
    ("by_parts", dict(factor=32.0, original_len=4096, low=1.0, high=32.0)),
    ("by_parts", dict(factor=8.0, original_len=8192, low=1.0, high=4.0, magnitude=1.0))])
def test_scaled_tables_at_far_positions(layout, scaling, kw):
    g = torch.Generator().manual_seed(9)
    x = torch.randn(200, 4, 64, generator=g)
    pos = torch.randint(0, 1_000_000, (200,), generator=g, dtype=torch.int32)
    table = api.rope_table(64, base=50000.0, scaling=scaling, **kw)
    magnitude = kw.pop("magnitude", 0.1 * np.log(kw["factor"]) + 1.0 if scaling == "by_parts" else 1.0)
    assert abs(table.magnitude - magnitude) < 1e-12
    freqs = oracle.rope_frequencies(64, 50000.0, scaling, **kw)
    out = api.mla_rope(x.cuda(), pos.cuda(), table, layout=layout)
    ref = oracle.rope_rotate(x.double().numpy(), pos.numpy(), freqs, layout, magnitude)
    tol = _bound(x.double().numpy(), ref, layout, magnitude, torch.float32)
    assert np.all(np.abs(_f64(out) - ref) <= tol)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_inverse_is_the_gradient(layout):
    """<g, R(x)> = <R'(g), x>, and along a difference: fp32, sums in double.  Each
    inner product is off by at most its elements' tolerance times the other factor."""
    g = torch.Generator().manual_seed(4)
    x, d = (torch.randn(33, 6, 64, generator=g).cuda() for _ in range(2))
    pos = torch.randint(0, 500_000, (33,), generator=g, dtype=torch.int32).cuda()
    table = api.rope_table(64, scaling="by_parts", factor=16.0, original_len=4096)
    y = api.mla_rope(x, pos, table, layout=layout)
    back = api.mla_rope(d, pos, table, layout=layout, inverse=True)
    lhs, rhs = (d.double() * y.double()).sum(), (back.double() * x.double()).sum()
    tol = 2 * 2.0 ** -20 * table.magnitude * 2 * (d.abs().double().sum() * x.abs().max())
    assert abs(float(lhs - rhs)) <= float(tol)
    # the map is linear: a difference along e gives the same product at any step
    e = torch.randn(33, 6, 64, generator=g).cuda()
    y2 = api.mla_rope(x + e, pos, table, layout=layout)
    lhs = (d.double() * (y2.double() - y.double())).sum()
    rhs = (back.double() * ((x + e).double() - x.double())).sum()
    assert abs(float(lhs - rhs)) <= 4 * float(tol)


def test_in_place_strided_and_out_views():
    g = torch.Generator().manual_seed(5)
    table = api.rope_table(64)
    pos = torch.arange(1000, 1037, dtype=torch.int32, device="cuda")
    base = torch.randn(37, 8, 192, generator=g).to(torch.bfloat16).cuda()
    want = api.mla_rope(base[..., 128:], pos, table)
    # in place inside the wider heads: the other 128 elements stay
    wide = base.clone()
    got = api.mla_rope(wide[..., 128:], pos, table, out=wide[..., 128:])
    assert got.data_ptr() == wide[..., 128:].data_ptr()
    assert torch.equal(wide[..., 128:], want) and torch.equal(wide[..., :128], base[..., :128])
    # heads before tokens, and an expanded (shared) head
    turned = base[..., 128:].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(api.mla_rope(turned, pos, table), want)
    one = base[:, :1, 128:]
    assert torch.equal(api.mla_rope(one.expand(37, 5, 64), pos, table),
                       api.mla_rope(one.contiguous(), pos, table).expand(37, 5, 64))
    # an output with its own strides and an odd address: element by element
    holder = torch.full((37, 8, 67), 7.0, dtype=torch.bfloat16, device="cuda")
    api.mla_rope(base[..., 128:], pos, table, out=holder[..., 1:65])
    assert torch.equal(holder[..., 1:65], want)
    assert bool((holder[..., 0] == 7).all()) and bool((holder[..., 65:] == 7).all())
    # nothing to do
    assert api.mla_rope(base[:0, :, 128:], pos[:0], table).shape == (0, 8, 64)


def test_non_finite_values_stay_in_their_pairs():
    x = torch.ones(1, 1, 64, device="cuda")
    x[0, 0, 3] = float("nan")
    x[0, 0, 40] = float("inf")
    out = api.mla_rope(x, torch.tensor([5], dtype=torch.int32, device="cuda"), api.rope_table(64))
    bad = ~torch.isfinite(out[0, 0]).cpu()
    assert sorted(torch.nonzero(bad).flatten().tolist()) == [3, 8, 35, 40]


def _pool(w, fp8, poison=True):
    return (inputs.make_slab_e4m3 if fp8 else inputs.make_slab)(w, "cpu", poison_nan=poison)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("lengths,n_new,H,own,pad", [
    ([1000, 2000, 3100], 1, 16, False, 0), ([1536, 1537, 4608], 4, 64, True, 0),
    ([700] * 37, 2, 3, True, 32), ([4000], 1601, 5, False, 0), ([9, 10], 3, 0, True, 0)])
def test_append_rotates_and_places(fp8, layout, lengths, n_new, H, own, pad):
    w = inputs.custom_workload(lengths, 1, 16, seed=3, page_stride=PT * ROW + pad)
    g = torch.Generator().manual_seed(11)
    rows = w.num_reqs * n_new
    lat = torch.randn(rows, 512, generator=g).to(torch.bfloat16)
    rope = torch.randn(rows, 64, generator=g).to(torch.bfloat16)
    q = torch.randn(rows, max(H, 1), 192, generator=g).to(torch.bfloat16).cuda()[..., 128:]
    at = (np.asarray(w.seq_lens)[:, None] - n_new + np.arange(n_new)[None]).reshape(-1)
    pos = at + 612_345 if own else at
    table = api.rope_table(64, base=50000.0, scaling="linear", factor=4.0, magnitude=1.25)
    freqs = oracle.rope_frequencies(64, 50000.0, "linear", 4.0)
    slab = _pool(w, fp8)
    dev = slab.cuda()
    ids = torch.as_tensor(w.page_table, device="cuda")
    lens = torch.as_tensor(w.seq_lens, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(positions=torch.as_tensor(pos.astype(np.int32), device="cuda") if own else None,
              layout=layout, q_rope=q if H else None, status=status)
    scale = inputs.KV_SCALE_E4M3
    if fp8:
        q_out = api.mla_kv_append_rope_fp8(lat.cuda(), rope.cuda(), dev, ids, lens, n_new, table,
                                           kv_scale=scale, **kw)
    else:
        q_out = api.mla_kv_append_rope(lat.cuda(), rope.cuda(), dev, ids, lens, n_new, table, **kw)
    assert int(status.item()) == 0
    got = dev.cpu().view(torch.uint8 if fp8 else torch.int16).numpy()
    want = np.array(slab.view(torch.uint8 if fp8 else torch.int16).numpy())
    ref = oracle.rope_rotate(rope.double().numpy()[:, None], pos, freqs, layout, 1.25)[:, 0]
    bound = _bound(rope.double().numpy()[:, None], ref[:, None], layout, 1.25, torch.float32)[:, 0]
    for i in range(rows):
        r, p = i // n_new, int(at[i])
        page, row = int(w.page_table[r, p // PT]), slice(p % PT * ROW, (p % PT + 1) * ROW)
        have = got[page, row]
        if fp8:
            assert np.array_equal(have[:512], oracle.e4m3_encode(
                (lat[i].float().numpy() / np.float32(scale)).astype(np.float64)))
            v = oracle.e4m3_decode(have[512:]) * scale
            # E4M3 rounds by 2^-4 relative, or half its smallest step 2^-10
            clipped = np.clip(ref[i], -448 * scale, 448 * scale)
            tol = bound[i] + np.maximum(2.0 ** -4 * (np.abs(clipped) + bound[i]), 2.0 ** -10 * scale)
            assert np.all(np.abs(v - clipped) <= tol * (1 + 2.0 ** -20))
        else:
            assert np.array_equal(have[:512], lat[i].view(torch.int16).numpy())
            v = torch.from_numpy(have[512:].copy()).view(torch.bfloat16).double().numpy()
            assert np.all(np.abs(v - ref[i]) <= bound[i] + 2.0 ** -8 * (np.abs(ref[i]) + bound[i]))
        want[page, row] = have
    assert np.array_equal(got, want), "something besides the new rows was written"
    if H:
        ref = oracle.rope_rotate(_f64(q), pos, freqs, layout, 1.25)
        assert q_out.is_contiguous()
        assert np.all(np.abs(_f64(q_out) - ref) <=
                      _bound(_f64(q), ref, layout, 1.25, torch.bfloat16))
    else:
        assert q_out is None


def test_unrotated_positions_equal_the_plain_append():
    """At position 0 the rotation is the identity: bit for bit mla_kv_append."""
    w = inputs.custom_workload([1700, 900], 1, 16, seed=6)
    g = torch.Generator().manual_seed(2)
    lat = torch.randn(8, 512, generator=g).to(torch.bfloat16).cuda()
    rope = torch.randn(8, 64, generator=g).to(torch.bfloat16).cuda()
    ids, lens = (torch.as_tensor(a, device="cuda") for a in (w.page_table, w.seq_lens))
    zero = torch.zeros(8, dtype=torch.int32, device="cuda")
    for fp8 in (False, True):
        a, b = _pool(w, fp8, False).cuda(), _pool(w, fp8, False).cuda()
        if fp8:
            api.mla_kv_append_fp8(lat, rope, a, ids, lens, 4, kv_scale=0.0371)
            api.mla_kv_append_rope_fp8(lat, rope, b, ids, lens, 4, api.rope_table(64),
                                       positions=zero, kv_scale=0.0371)
        else:
            api.mla_kv_append(lat, rope, a, ids, lens, 4)
            api.mla_kv_append_rope(lat, rope, b, ids, lens, 4, api.rope_table(64), positions=zero)
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_rows_are_skipped_and_reported(fp8):
    w = inputs.custom_workload([3000, 2000], 1, 16, seed=4, spare_pages=2)
    g = torch.Generator().manual_seed(2)
    lat = torch.randn(4, 512, generator=g).to(torch.bfloat16).cuda()
    rope = torch.randn(4, 64, generator=g).to(torch.bfloat16).cuda()
    table = api.rope_table(64)

    def run(ids, lens, before):
        dev, status = before.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        args = (lat, rope, dev, torch.as_tensor(ids, device="cuda"),
                torch.as_tensor(np.asarray(lens, dtype=np.int32), device="cuda"), 2, table)
        if fp8:
            api.mla_kv_append_rope_fp8(*args, kv_scale=0.05, status=status)
        else:
            api.mla_kv_append_rope(*args, status=status)
        changed = (dev.view(torch.uint8) != before.view(torch.uint8)).view(
            dev.shape[0], -1).any(1)
        return int(status.item()), torch.nonzero(changed).flatten().tolist()

    before = _pool(w, fp8, False).cuda()
    code, pages = run(w.page_table, [3000, 1], before)     # one row before the history
    assert code == 32 and pages == sorted({int(w.page_table[0, 1]), int(w.page_table[1, 0])})
    ids = np.array(w.page_table)
    ids[0, 1] = w.num_pages                                # outside the pool
    code, pages = run(ids, w.seq_lens, before)
    assert code == 33 and pages == [int(ids[1, 1])]
    ids[0, 1] = -5
    code, pages = run(ids, w.seq_lens, before)
    assert code == 33 and pages == [int(ids[1, 1])]
    # past the table's row
    code, pages = run(np.ascontiguousarray(w.page_table[:, :1]), [1000, 1537], before)
    assert code == 33 and pages == sorted({int(w.page_table[0, 0]), int(w.page_table[1, 0])})


def test_replayed_graph_on_another_stream():
    """Captured once, replayed on new positions and data, on a stream of its own."""
    w = inputs.custom_workload([1600, 40], 1, 16, seed=8)
    g = torch.Generator().manual_seed(7)
    table = api.rope_table(64)
    slab = _pool(w, False, False).cuda()
    ids, lens = (torch.as_tensor(a, device="cuda") for a in (w.page_table, w.seq_lens))
    lat = torch.randn(2, 512, generator=g).to(torch.bfloat16).cuda()
    rope = torch.randn(2, 64, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(2, 4, 64, generator=g).to(torch.bfloat16).cuda()
    q_out, pos = torch.empty_like(q), torch.zeros(2, dtype=torch.int32, device="cuda")

    def step(pool, out, stream=None):
        api.mla_kv_append_rope(lat, rope, pool, ids, lens, 1, table, positions=pos, q_rope=q,
                               q_out=out, stream=stream)
    step(slab, q_out)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        step(slab, q_out)
    pos.copy_(torch.tensor([77_000, 3], dtype=torch.int32))
    rope.copy_(torch.randn(2, 64, generator=g).to(torch.bfloat16))
    other, want = slab.clone(), torch.empty_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.replay()
    step(other, want, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(q_out, want) and torch.equal(slab, other)


def test_front_end_refusals():
    table = api.rope_table(64)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    bad = [
        lambda: api.mla_rope(x[..., :32], pos, table),
        lambda: api.mla_rope(x, pos.long(), table),
        lambda: api.mla_rope(x, pos[:3], table),
        lambda: api.mla_rope(x, pos.cpu(), table),
        lambda: api.mla_rope(x.double(), pos, table),
        lambda: api.mla_rope(x, pos, table, layout="rows"),
        lambda: api.mla_rope(x, pos, table, out=x.float()),
        lambda: api.mla_rope(x[1:], pos[1:], table, out=x[:3]),           # overlapping
        lambda: api.mla_rope(x, pos, table, out=x[:, :1].expand(4, 2, 64)),
        lambda: api.mla_rope(x.transpose(1, 2).contiguous().transpose(1, 2), pos, table),
    ]
    lat = torch.zeros(2, 512, dtype=torch.bfloat16, device="cuda")
    slab = torch.zeros(2, PT * ROW, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")

    def append(t=table, **kw):
        return api.mla_kv_append_rope(lat, lat[:, :64].contiguous(), slab, ids, lens, 1, t, **kw)
    bad += [
        lambda: append(api.rope_table(32)),
        lambda: append(positions=pos),
        lambda: append(q_rope=x),
        lambda: append(q_out=x[:2]),
        lambda: append(q_rope=x[:2], q_out=x[:2]),
        lambda: append(layout="pairs"),
        lambda: append(status=torch.zeros(1, device="cuda")),
        lambda: api.mla_kv_append_rope_fp8(lat, lat[:, :64].contiguous(), slab.view(torch.uint8),
                                           ids, lens, 1, table, kv_scale=0.0),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
