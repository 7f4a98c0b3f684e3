"""The norm, the cache and the batch at their edges, as far as the host decides:
the objects take tensors of the CPU here, and no call reaches the library."""
import os
import types

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_19_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from mixture_experts_layer_19_amd import build
        build.build()
    binding.lib()
    return binding


@pytest.fixture
def block(B, monkeypatch):
    from mixture_experts_layer_19_amd import block
    monkeypatch.setattr(block, "_device", lambda t: t.device)
    return block


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def objects(block):
    batch = block.KVBatch(i32(3, 5), i32(4), i32(3), rows=10, max_rows=4)
    cache = block.PagedKVCache(2, 64, 4, 16, dtype="mxfp8", device="cpu")
    return batch, cache, block.RMSNorm(torch.ones(64), quant="mxfp8")


def test_counts_stay_those_that_the_library_was_given(block):
    """Assigning one would leave the old one in the C structs, which the kernels
    count by, beside tensors of the new shape."""
    batch, cache, norm = objects(block)
    for obj, names in ((batch, ("seqs", "rows", "max_rows", "c")),
                       (cache, ("kv_heads", "head_dim", "num_pages", "page_size", "c")), (norm, ("hidden",))):
        for name in names:
            was = getattr(obj, name)
            for other in (2, 1000):
                with pytest.raises(AttributeError):
                    setattr(obj, name, other if was != other else other + 1)
            assert getattr(obj, name) is was
    for obj, name, other in ((cache, "dtype", "bf16"), (cache, "act_dtype", torch.float32),
                             (cache, "device", torch.device("cuda", 0)), (batch, "device", torch.device("cuda", 0)),
                             (norm, "quant", "none"), (norm, "dtype", torch.bfloat16),
                             (norm, "device", torch.device("cuda", 0))):
        with pytest.raises(AttributeError):
            setattr(obj, name, other)
    assert (batch.c.rows, batch.c.max_rows, batch.c.seqs) == (batch.rows, batch.max_rows, batch.seqs) == (10, 4, 3)
    batch.kv_len += 1                                    # in place
    assert batch.kv_len.tolist() == [1, 1, 1]


P = 1 << 20          # a pointer that is aligned and never read


def cache_of(B, **kw):
    return B.MoeKvCache(**dict(dict(k=P, v=P, k_scale=P, v_scale=P, num_pages=10, page_size=16, kv_heads=2, head_dim=128,
                                    dtype=B.MOE_MXFP8), **kw))


def batch_of(B, **kw):
    return B.MoeKvBatch(**dict(dict(page_table=P, row_offsets=P, kv_len=P, seqs=3, max_pages=200, rows=6, max_rows=2),
                               **kw))


def test_sinks_that_cover_the_table_hide_nothing(B):
    """Their number does not overflow: the cut, and its workspace, are those without a window."""
    for max_pages in (200, 100000):
        for rows, max_rows in ((6, 2), (600, 300)):
            c, b = cache_of(B), batch_of(B, max_pages=max_pages, rows=rows, max_rows=max_rows)
            whole = B.moe_attention_workspace_bytes(c, b, 4, 0, 0)
            assert whole > 0
            for sinks in (16 * max_pages, 2 ** 31 - 128, 2 ** 31 - 1):
                assert B.moe_attention_workspace_bytes(c, b, 4, 100, sinks) == whole


@pytest.mark.parametrize("c,b,heads", [
    # a workgroup a unit; pieces of cut units to join; tiles of 256 rows
    (dict(kv_heads=8), dict(seqs=1 << 21, rows=1 << 21, max_rows=1, max_pages=2), 8),
    (dict(kv_heads=8), dict(seqs=1 << 21, rows=1 << 21, max_rows=1, max_pages=100), 8),
    (dict(kv_heads=8, head_dim=256), dict(seqs=1 << 19, rows=1 << 20, max_rows=2, max_pages=100), 64),
    (dict(kv_heads=8), dict(seqs=1 << 20, rows=1 << 21, max_rows=2, max_pages=2), 512)])
def test_attention_refuses_more_units_than_a_launch_holds(B, c, b, heads):
    """A launch of 2^32 threads and more would run part of them."""
    with pytest.raises(B.MoeError) as ei:
        B.moe_attention(cache_of(B, **c), batch_of(B, **b), P, 512 * heads, 512, heads, 0.1, 0, 0, P, P, 1 << 50)
    assert ei.value.status == B.MOE_ERR_UNSUPPORTED


ONCE = r"""
#include "once_per_device.hpp"
#include <assert.h>
#include <thread>
#include <vector>
int main() {
  moe::OncePerDevice once;
  int calls[80] = {0};
  auto call = [&](int d, int result) { return once(d, [&] { ++calls[d]; return result; }); };
  assert(call(0, 0) == 0 && call(0, 0) == 0 && calls[0] == 1);      // set once
  assert(call(1, 0) == 0 && calls[1] == 1 && calls[0] == 1);        // another device: of its own
  assert(call(2, 7) == 7 && call(2, 7) == 7 && calls[2] == 2);      // a failure is not kept
  assert(call(2, 0) == 0 && call(2, 7) == 0 && calls[2] == 3);
  assert(call(63, 0) == 0 && call(63, 1) == 0 && calls[63] == 1);
  assert(call(70, 0) == 0 && call(70, 0) == 0 && calls[70] == 2);   // past the mask: every time
  moe::OncePerDevice other;
  std::atomic<int> n{0};
  std::vector<std::thread> t;
  for (int i = 0; i < 16; ++i)
    t.emplace_back([&, i] { for (int k = 0; k < 1000; ++k) other(i % 4, [&] { ++n; return 0; }); });
  for (auto &x : t) x.join();
  assert(n >= 4 && n <= 16);
  return 0;
}
"""


def test_a_kernels_setting_is_made_on_every_device(tmp_path):
    """The limit of dynamic LDS belongs to a kernel on one device."""
    import subprocess
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_19_amd", "csrc")
    src = tmp_path / "once.cpp"
    src.write_text(ONCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", csrc, str(src), "-o", str(tmp_path / "once")], check=True)
    subprocess.run([str(tmp_path / "once")], check=True, timeout=60)
    for name in ("attn_rows.hip", "attn_tile.hip"):
        text = open(os.path.join(csrc, name)).read()
        assert "hipFuncSetAttribute" not in text and "allow_lds(once" in text


def test_streams_of_another_device_are_refused(block):
    """The call would have run on that device's current stream, beside the one given."""
    batch, cache, norm = objects(block)
    for index in (1, 7):
        other = types.SimpleNamespace(device_index=index, device=torch.device("cuda", index))
        for call in (lambda: norm(torch.ones(2, 64), stream=other),
                     lambda: cache.read(batch, stream=other),
                     lambda: cache.write(batch, *(torch.zeros(10, 2, 64, dtype=torch.bfloat16),) * 2, stream=other),
                     lambda: cache.attention(batch, torch.zeros(10, 4, 64, dtype=torch.bfloat16), stream=other)):
            with pytest.raises(ValueError, match="another device"):
                call()


def test_counts_past_32_bits_are_refused(block):
    """Passing one on would cut it to its low 32 bits: 2^32 + 5 rows would be 5."""
    _, cache, norm = objects(block)
    with pytest.raises(ValueError, match="2.31"):
        norm(torch.ones(1, 64).expand(2 ** 32 + 5, 64))
    with pytest.raises(ValueError, match="2.31"):
        norm(torch.ones(1, 64).expand(2 ** 31, 64))
    for rows in (2 ** 31, 2 ** 32 + 5):
        with pytest.raises(ValueError, match="2.31"):
            block.KVBatch(i32(3, 5), i32(4), i32(3), rows=rows)
    for kw in (dict(kv_heads=2 ** 32 + 1), dict(num_pages=2 ** 32 + 1)):
        with pytest.raises(ValueError, match="2.31"):
            block.PagedKVCache(**dict(dict(kv_heads=1, head_dim=64, num_pages=1, page_size=1, device="meta"), **kw))


def test_cache_kernels_keep_their_pieces_in_registers(tmp_path):
    """The pieces in flight are in registers: beside the rows' places (4 bytes each of 4
    or 8 rows) the compiler gives the kernels neither LDS nor scratch memory."""
    import re
    import subprocess
    from mixture_experts_layer_19_amd import build
    cmd = [build._hipcc(), "--offload-arch=" + build.ARCH, "-O3", "-std=c++17", "-fPIC", "-Xclang", "-target-feature",
           "-Xclang", "-packed-fp32-ops", "-I", os.path.join(build.ROOT, "include"), "--cuda-device-only",
           "-Rpass-analysis=kernel-resource-usage", "-c", os.path.join(build.CSRC, "kv.hip"), "-o", str(tmp_path / "kv.o")]
    text = subprocess.run(cmd, check=True, capture_output=True, text=True, timeout=300).stderr
    names = re.findall(r"Function Name: (\S+)", text)
    lds = [int(n) for n in re.findall(r"LDS Size \[bytes/block\]: (\d+)", text)]
    scratch = [int(n) for n in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", text)]
    assert len(names) == len(lds) == len(scratch) == 12
    for name, n, s in zip(names, lds, scratch):
        assert n <= 32 and s == 0, name
