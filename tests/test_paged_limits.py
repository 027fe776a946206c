"""Sizes at the ends of what the paged attention operators accept: numbers beyond 32 bits are
refused and never taken modulo 2^32."""
import numpy as np
import pytest

WRAPS = 2 ** 32 + 4                                # 4, taken modulo 2^32


@pytest.mark.parametrize("at, name", [(0, "rows"), (5, "batch"), (6, "width"), (7, "max_len")])
def test_sizes_beyond_32_bits(at, name):
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    sizes = [4, 8, (100, 2, 64, 128), torch.bfloat16, None, 4, 20, 40]
    assert ops._paged(*sizes).max_len == 40
    for big in (WRAPS, 2 ** 31):
        sizes[at] = big
        with pytest.raises(ValueError, match=name):
            ops._paged(*sizes)


def test_cache_sizes_beyond_32_bits():
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    for shape in ((WRAPS, 2, 64, 128), (100, WRAPS, 64, 128), (100, 2, WRAPS, 128), (100, 2, 64, WRAPS)):
        with pytest.raises(ValueError, match="32 bits"):
            ops._paged(4, 8, shape, torch.bfloat16)
    with pytest.raises(ValueError, match="32 bits"):
        ops.paged_workspace_bytes(ops._paged(4, 8, (100, 2, 64, 128), torch.bfloat16), WRAPS)


def test_bookkeeping_sizes_beyond_32_bits():
    """Whatever the tensors' device: the sizes come first."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    lens, pos = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    table, ring = torch.zeros((2, 1), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    wide, long, many = table.expand(2, WRAPS), ring.expand(WRAPS), table[:1].expand(WRAPS, 1)
    for kw, name in ((dict(page=2 ** 32 + 16), "page"), (dict(rows=WRAPS), "rows"), (dict(table=wide), "width"),
                     (dict(free_list=long), "free_list"), (dict(table=many), "batch")):
        call = {**dict(lens=lens, table=table, free_list=ring, free_pos=pos, page=16, rows=4), **kw}
        with pytest.raises(ValueError, match=name):
            ops.paged_plan(add=lens, **call)
        if name != "rows":
            del call["rows"]
            with pytest.raises(ValueError, match=name):
                ops.paged_release(done=lens.byte(), **call)


def test_select_counts_beyond_32_bits():
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    q, codes = torch.zeros((1, 2, 64)), torch.zeros((3, 1, 64), dtype=torch.int8)
    table, one = torch.zeros((1, 3), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for kw in (dict(n_sink=2 ** 32), dict(n_local=2 ** 32 + 1), dict(n_blocks=WRAPS)):
        with pytest.raises(ValueError, match=next(iter(kw))):
            ops.paged_select(**{**dict(q=q, codes=codes, code_scale=torch.ones((3, 1)), table=table, row_len=one, page=16, n_blocks=4), **kw})


@pytest.mark.gpu
def test_refused_on_the_device():
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    i32 = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()
    q, cache = torch.zeros((1, 2, 64), device="cuda"), torch.zeros((3, 1, 16, 64), device="cuda")
    table, length = i32([[0, 1, 2]]), i32([40])
    codes, scale = torch.zeros((3, 1, 64), dtype=torch.int8, device="cuda"), torch.ones((3, 1), device="cuda")
    for kw in (dict(max_len=WRAPS), dict(max_len=torch.tensor(WRAPS))):
        with pytest.raises(ValueError, match="max_len"):
            ops.paged_attend(q, cache, cache, table, length, **kw)
        with pytest.raises(ValueError, match="max_len"):
            ops.paged_select(q, codes, scale, table, length, 16, 2, **kw)
    with pytest.raises(ValueError, match="page"):
        ops.paged_select(q, codes, scale, table, length, 2 ** 32 + 16, 2)


def _fake_plan(batch, rows):
    import ctypes
    from gated_deltanet_prefill_chunkwise_amd import ops
    fake = [ctypes.c_void_p(0x1000)] * 13           # never dereferenced: refused, or no device here
    L = ops.lib()
    return (L.sgdn_paged_plan(batch, 16, 4, rows, 9, *fake, None), L.sgdn_paged_release(batch, 16, 4, 9, *fake[:7], None))


@pytest.mark.parametrize("batch, rows", [(2 ** 31 - 1024, 5), (2 ** 31 - 1, 5), (5, 2 ** 31 - 1024), (5, 2 ** 31 - 1)])
def test_bookkeeping_of_more_than_its_counters_hold(batch, rows):
    """Kernels count requests and rows in steps of up to 1024: the last step has to end below 2^31."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("checks of arguments, on hosts without a device")
    plan, release = _fake_plan(batch, rows)
    assert plan == -2 and (release == -2) == (batch > 5)


def test_write_of_more_rows_than_a_launch_holds():
    """16 rows a workgroup of 256: 2^28 - 15 rows and more would round up to 2^32 threads."""
    import ctypes
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    if torch.cuda.is_available():
        pytest.skip("checks of arguments, on hosts without a device")
    fake = ctypes.c_void_p(0x1000)
    for rows, status in ((2 ** 28 - 1, -2), (2 ** 28 - 15, -2), (2 ** 28 - 16, -1)):   # enough room: the next check
        shape = ops.Paged(rows, 1, 1, 1, 64, 16, 100, 1, 0, 1, 1)
        k = None if status == -1 else fake
        assert ops.lib().sgdn_paged_write(ctypes.byref(shape), k, fake, 64, 64, fake, fake, fake, None, None, None) == status
