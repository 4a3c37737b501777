"""Blocks beyond the first 4 GiB of a pool: the same blocks at the end of a pool of
4.6 GB and in a small one give the same bits."""
import numpy as np
import pytest

from tests._gpu import check_device_error, dev, torch_cuda
from tests._score_mod import queries, slopes_of

pytestmark = pytest.mark.gpu

HK, D, FAR = 8, 128, 140_000


@pytest.fixture(scope="module")
def pk(capi):
    torch_cuda()
    import paged_kv_cache_59_gb300 as m
    m.pa_get_device_error()
    return m


@pytest.mark.parametrize("kind", ["bf16", "block"])
def test_far_blocks(pk, kind):
    torch = torch_cuda()
    nb = FAR if kind == "bf16" else 2 * FAR
    gen = torch.Generator(device="cuda").manual_seed(5)
    near = [torch.randn((12, HK, 16, D), generator=gen, device="cuda") for _ in range(2)]
    if kind == "bf16":
        near, scales = [x.to(torch.bfloat16).view(torch.int16) for x in near], None
    else:
        near = [x.to(torch.float8_e4m3fn).view(torch.uint8) for x in near]
        scales = [torch.exp2(torch.randint(-3, 3, (12, HK), generator=gen, device="cuda").float()) for _ in range(2)]
    ids = torch.arange(nb - 12, nb, device="cuda").flip(0)
    results = []
    for far in (False, True):
        if far:
            pools = [torch.zeros((nb, HK, 16, D), dtype=near[0].dtype, device="cuda") for _ in range(2)]
            assert pools[0].numel() * pools[0].element_size() > 2 ** 32
            for p, x in zip(pools, near):
                p[ids] = x
            sc = None if scales is None else [torch.ones((nb, HK), device="cuda") for _ in range(2)]
            for a, b in zip(sc or [], scales or []):
                a[ids] = b
            order = ids
        else:
            pools, order = [x.clone() for x in near], torch.arange(12, device="cuda")
            sc = None if scales is None else [x.clone() for x in scales]
        more = {} if sc is None else dict(k_scale=sc[0], v_scale=sc[1])
        tables = order[None].int().contiguous()
        keep = dev(np.sort(np.random.default_rng(1).choice(190, 120, replace=False)).astype(np.int32))
        pk.pa_compact_blocks(*pools, tables, keep, dev(np.array([0, 120], np.int32)), **more)
        q = dev(queries(3, 40, 32, D))
        out, one = torch.zeros_like(q), torch.zeros_like(q[:1])
        ctx = dev(np.array([120], np.int32))
        mods = dict(softcap=30.0, alibi_slopes=dev(slopes_of(32)), **more)
        pk.pa_prefill_score_mod(out, q, *pools, tables, ctx, dev(np.array([0, 40], np.int32)), D ** -0.5, 40, splits=1, **mods)
        pk.pa_decode_score_mod(one, q[:1].contiguous(), *pools, tables, ctx, D ** -0.5, 120, **mods)
        torch.cuda.synchronize()
        results.append([out, one] + [p[order] for p in pools] + ([] if sc is None else [s[order] for s in sc]))
        del pools
    for a, b in zip(*results):
        assert torch.equal(a, b)
    check_device_error(0)
