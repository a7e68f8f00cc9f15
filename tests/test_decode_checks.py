"""More argument checks of the decoding step's calls, without a GPU: nothing here reaches a kernel."""
import ctypes

import pytest

from token_level_top_gb300 import build, moe

FAKE = 0x7f0000000000  # never dereferenced: every call below is refused
R = ctypes.byref


@pytest.fixture(scope="module")
def L():
    build.build()
    return moe.lib()


def _cache(e4m3=False, **kw):
    d = dict(k=FAKE, v=FAKE, k_exp=FAKE if e4m3 else None, v_exp=FAKE if e4m3 else None, type=1 if e4m3 else 0, n_pages=4,
             page_size=16, n_kv_heads=2, head_dim=128, page_stride=4096, token_stride=128, head_stride=2048)
    d.update(kw)
    return moe.MoEKVCache(**d)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kw", [dict(page_stride=-4096), dict(token_stride=-128), dict(page_stride=-16), dict(token_stride=-2 ** 40)])
def test_negative_page_and_token_strides_are_refused(L, e4m3, kw):
    """By both calls that take a cache: the append would find no place for any token."""
    a = moe.MoEAppend(T=3, n_seqs=3, max_pages=2, n_heads=0, rot_dim=0, flags=0, pos=FAKE, seq=None, page_table=FAKE,
                      table_stride=2, phase=None, q=None, k=FAKE, v=FAKE, q_out=None, k_token_stride=256, k_head_stride=128,
                      v_token_stride=256, v_head_stride=128)
    assert L.moe_kv_append(R(_cache(e4m3, **kw)), R(a), None, None) == 2
    t = moe.MoEAttention(3, 4, 2, 0, 0.1, FAKE, FAKE, 2, FAKE, FAKE, None, 512, 128, 512, 128)
    n = L.moe_paged_attention_workspace_size(128)
    assert L.moe_paged_attention(R(_cache(e4m3, **kw)), R(t), ctypes.c_void_p(FAKE), n, None) == 2


def test_memory_of_another_kind_is_refused():
    """Status words and workspaces reach a kernel as addresses: host memory and too little of it are refused before."""
    import torch
    host = torch.zeros(64, dtype=torch.int32)
    for t in (host, host[:0], host.view(torch.uint8)[1:9], host[::2]):
        with pytest.raises(ValueError, match="status"):
            moe._memory(t, "status", 0)
    with pytest.raises(ValueError, match="current CUDA device"):
        moe._device(host, "k")
    with pytest.raises(ValueError, match="CUDA device 0"):
        moe._rows(host, "pos", 64, 0)
    # the last condition by itself: what get_device() says of host memory is -1
    assert moe._memory(host, "status", -1) == host.data_ptr()
    for t in (host[:0], host.view(torch.uint8)[1:9], host.view(torch.uint8)[:3], host[::2], host[:1].expand(64)):
        with pytest.raises(ValueError, match="status"):
            moe._memory(t, "status", -1)
