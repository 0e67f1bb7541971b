"""Host-side tests of the decoding step's operators' ABI (no GPU needed): structure
layout, and every refusal before any launch, in C and in Python."""
import ctypes as C
import math
import os
import subprocess

import pytest
import torch

from routed_moe_decode_router_gb300 import build as B
from routed_moe_decode_router_gb300 import native as N
from routed_moe_decode_router_gb300 import fp8_layer, ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 28      # a well-aligned address that no refused call may touch


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return N.lib()


def refused(fn, *a, status=1, text=""):
    with pytest.raises(N.MoeError) as e:
        fn(*a)
    assert e.value.status == status and text in str(e.value), str(e.value)


def test_struct_layout(tmp_path):
    structs = {"moeop_kv_cache": N.KvCache, "moeop_attend_config": N.AttendConfig,
               "moeop_verify_config": N.VerifyConfig}
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "moe_ops.h"', 'int main(void){']
    for c, py in structs.items():
        src.append('printf("%s %%zu\\n", sizeof(%s));' % (c, c))
        src += ['printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (c, f, c, f) for f, _ in py._fields_]
    src.append('printf("e4m3 %d\\n", MOEOP_E4M3);')
    (tmp_path / "l.c").write_text("\n".join(src + ["return 0;}"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o",
                    str(tmp_path / "l")], check=True)
    got = dict(line.split() for line in subprocess.run(
        [str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.splitlines())
    for c, py in structs.items():
        assert int(got[c]) == C.sizeof(py)
        for f, _ in py._fields_:
            assert int(got["%s.%s" % (c, f)]) == getattr(py, f).offset
    assert int(got["e4m3"]) == N.MOEOP_E4M3


def cache(**kw):
    """8 pages of 32 tokens, 2 heads of 64, e4m3: 32 KB of codes and 2 KB of scales."""
    d = dict(k=P, v=2 * P, k_scales=3 * P, v_scales=4 * P, k_stride=4096, v_stride=4096,
             k_scales_stride=64, v_scales_stride=64, pages=8, heads=2, page=32, dim=64,
             type=N.MOEOP_E4M3)
    d.update(kw)
    return N.KvCache(**d)


BAD_CACHES = [
    (dict(type=2), "type"), (dict(type=4), "type"), (dict(dim=32), "dim"), (dict(dim=96), "dim"),
    (dict(page=8), "page"), (dict(page=40), "page"), (dict(page=1040), "page"),
    (dict(heads=0), "heads"), (dict(heads=1025), "heads"), (dict(pages=0), "pages"),
    (dict(pages=1 << 27), "pages"), (dict(k=0), "aligned"), (dict(v=2 * P + 8), "aligned"),
    (dict(k_stride=4095), "strides"), (dict(v_stride=4100), "strides"),
    (dict(k_stride=1 << 41), "strides"), (dict(k_scales=0), "k_scales"),
    (dict(v_scales=4 * P + 4), "16-byte"), (dict(k_scales_stride=63), "scales"),
    (dict(v_scales_stride=66), "scales"), (dict(v=P), "two arrays"), (dict(v=P + 4096), "two arrays"),
    (dict(k_scales=2 * P + 256), "two arrays"), (dict(v_scales=3 * P), "two arrays"),
    (dict(k_stride=8192, v_stride=8192, v=P + 2048), "two arrays"),
    (dict(type=0), "no scales"), (dict(type=0, k_scales=0), "no scales")]


@pytest.mark.parametrize("kw,text", BAD_CACHES)
def test_cache_refusals(kw, text):
    refused(N.moeop_kv_write, cache(**kw), 5 * P, 128, 6 * P, 128, 0, 7 * P, 4, text=text)
    refused(N.moeop_kv_read, cache(**kw), 7 * P, 4, 5 * P, 6 * P, 0, text=text)
    refused(N.moeop_attend_paged, config(), cache(**kw), *attend_args(), text=text)


def test_keys_and_values_may_lie_in_turn():
    turn = cache(k_stride=8192, v_stride=8192, v=P + 4096)
    refused(N.moeop_kv_write, turn, 0, 128, 6 * P, 128, 0, 7 * P, 4, text="NULL")   # nothing before
    refused(N.moeop_kv_write, turn, 0, 128, 6 * P, 128, 0, 7 * P, 4, text="aligned")


@pytest.mark.parametrize("kw,text", [
    (dict(dtype=3), "dtype"), (dict(dtype=-1), "dtype"), (dict(tokens=-1), "tokens"),
    (dict(tokens=(1 << 29) + 1), "tokens"), (dict(k=0), "NULL"), (dict(v=6 * P + 2), "aligned"),
    (dict(slots=0), "slots"), (dict(slots=7 * P + 2), "slots"), (dict(ks=127), "strides"),
    (dict(vs=132), "strides"), (dict(dtype=2, ks=130), "strides"), (dict(k=P), "overlaps"),
    (dict(v=2 * P + 32752), "overlaps"), (dict(slots=3 * P + 2044), "overlaps")])
def test_write_refusals(kw, text):
    d = dict(k=5 * P, ks=128, v=6 * P, vs=128, dtype=0, slots=7 * P, tokens=4)
    d.update(kw)
    refused(N.moeop_kv_write, cache(), *d.values(), text=text)


def test_a_cache_of_16_bits_takes_its_own_type():
    half = cache(type=N.MOEOP_FP16, k_scales=0, v_scales=0)
    refused(N.moeop_kv_write, half, 5 * P, 128, 6 * P, 128, N.MOEOP_BF16, 7 * P, 4, text="own type")
    refused(N.moeop_attend_paged, config(), half, *attend_args(), text="own type")


@pytest.mark.parametrize("kw,text", [
    (dict(slots=0), "slots"), (dict(tokens=-2), "tokens"), (dict(k=0), "NULL"),
    (dict(v=6 * P + 8), "aligned"), (dict(dtype=3), "dtype"), (dict(v=5 * P + 512), "overlap"),
    (dict(k=P + 16), "overlap"), (dict(v=4 * P), "overlap"), (dict(k=7 * P), "overlap")])
def test_read_refusals(kw, text):
    d = dict(slots=7 * P, tokens=4, k=5 * P, v=6 * P, dtype=0)
    d.update(kw)
    refused(N.moeop_kv_read, cache(), *d.values(), text=text)


def config(**kw):
    d = dict(batch=3, rows=2, q_heads=8, width=4, window=0, scale=0.125, dtype=0)
    d.update(kw)
    return N.AttendConfig(**d)


def attend_args(**kw):
    d = dict(q=5 * P, qb=1024, qr=512, table=6 * P, ts=4, lengths=7 * P, out=8 * P, ws=9 * P,
             n=1 << 27)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,text", [
    (dict(batch=-1), "batch"), (dict(batch=2049), "batch"), (dict(rows=0), "rows"),
    (dict(rows=65), "rows"), (dict(q_heads=0), "q_heads"), (dict(q_heads=7), "q_heads"),
    (dict(q_heads=258, rows=2), "q_heads"), (dict(width=0), "width"), (dict(width=1 << 26), "width"),
    (dict(batch=2048, width=1 << 20), "batch"), (dict(window=-1), "window"),
    (dict(scale=math.inf), "scale"), (dict(scale=math.nan), "scale"), (dict(dtype=2), "dtype"),
    (dict(dtype=3), "dtype")])
def test_attention_configurations_refused(kw, text):
    refused(N.moeop_attend_paged, config(**kw), cache(), *attend_args(), text=text)


@pytest.mark.parametrize("kw,status,text", [
    (dict(q=0), 1, "q and out"), (dict(q=5 * P + 8), 1, "aligned"), (dict(out=8 * P + 2), 1, "aligned"),
    (dict(table=0), 1, "table"), (dict(lengths=7 * P + 1), 1, "lengths"), (dict(qr=511), 1, "strides"),
    (dict(qb=1028), 1, "strides"), (dict(ts=3), 1, "table"), (dict(ws=0), 3, "NULL"),
    (dict(ws=9 * P + 128), 3, "256"), (dict(n=5000), 3, "needs"), (dict(out=5 * P), 1, "out overlaps"),
    (dict(out=P), 1, "out overlaps"), (dict(out=9 * P), 1, "out overlaps"),
    (dict(ws=4 * P), 1, "workspace overlaps"), (dict(lengths=9 * P), 1, "workspace overlaps")])
def test_attention_refusals(kw, status, text):
    refused(N.moeop_attend_paged, config(), cache(), *attend_args(**kw), status=status, text=text)


@pytest.mark.parametrize("a", [(-1, 1, 8, 2, 64), (2049, 1, 8, 2, 64), (1, 0, 8, 2, 64), (1, 65, 8, 8, 64),
                               (1, 1, 9, 2, 64), (1, 1, 8, 0, 64), (1, 1, 8, 2, 65), (1, 2, 258, 2, 64)])
def test_workspaces_refused(a):
    refused(N.moeop_attend_workspace_size, *a)


def test_workspace_sizes():
    size = N.moeop_attend_workspace_size
    assert size(0, 1, 8, 8, 64) == size(2048, 1, 8, 8, 64) > 0      # not a matter of the batch
    assert size(1, 1, 64, 8, 128) < size(1, 4, 64, 8, 128)
    assert all(size(1, r, 64, 8, d) < 64 << 20 for r in (1, 8, 32) for d in (64, 128, 256))
    refused(N.moeop_attend_workspace_init, 0, 1 << 20, status=3, text="NULL")
    refused(N.moeop_attend_workspace_init, P + 16, 1 << 20, status=3, text="256")
    refused(N.moeop_attend_workspace_init, P, 100, status=3, text="at least")


def verify_args(**kw):
    d = dict(draft=P, target=2 * P, probs=3 * P, u=4 * P, s=5 * P, tokens=6 * P, accepted=7 * P)
    d.update(kw)
    return list(d.values())


def verify_cfg(**kw):
    d = dict(batch=2, drafts=3, vocab=100, target_stride=100, draft_stride=100)
    d.update(kw)
    return N.VerifyConfig(**d)


@pytest.mark.parametrize("kw,text", [
    (dict(batch=-1), "batch"), (dict(batch=65536), "batch"), (dict(drafts=-1), "drafts"),
    (dict(drafts=32), "drafts"), (dict(vocab=0), "vocab"), (dict(vocab=(1 << 19) + 1), "vocab"),
    (dict(target_stride=99), "stride"), (dict(draft_stride=99), "stride")])
def test_verify_configurations_refused(kw, text):
    refused(N.moeop_verify_draft, verify_cfg(**kw), *verify_args(), text=text)


@pytest.mark.parametrize("kw,text", [
    (dict(draft=0), "NULL"), (dict(target=0), "NULL"), (dict(target=2 * P + 2), "aligned"),
    (dict(probs=3 * P + 1), "aligned"), (dict(u=0), "NULL"), (dict(s=0), "NULL"),
    (dict(tokens=0), "NULL"), (dict(accepted=7 * P + 2), "aligned"), (dict(tokens=7 * P), "overlap"),
    (dict(tokens=2 * P), "overlap"), (dict(accepted=3 * P + 396), "overlap"), (dict(tokens=P), "overlap"),
    (dict(accepted=5 * P), "overlap")])
def test_verify_refusals(kw, text):
    refused(N.moeop_verify_draft, verify_cfg(), *verify_args(**kw), text=text)


def test_empty_calls_touch_nothing():
    N.moeop_kv_write(cache(), 0, 0, 0, 0, 0, 0, 0)
    N.moeop_kv_read(cache(), 0, 0, 0, 0, 0)
    N.moeop_attend_paged(config(batch=0), cache(), 0, 0, 0, 0, 0, 0, 0, 0, 0)
    N.moeop_verify_draft(verify_cfg(batch=0), 0, 0, 0, 0, 0, 0, 0)


def test_python_refuses_host_tensors_before_the_library():
    host = ops.KvCache(torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16),
                       torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16))
    k, i = torch.zeros(1, 1, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    u = torch.zeros(1, 1)
    for call in (lambda: ops.kv_write(host, k, k, i), lambda: ops.kv_read(host, i),
                 lambda: ops.attend_paged(k, host, i[None], i),
                 lambda: ops.verify_draft(i[None], torch.zeros(1, 2, 5), u, u[0])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        ops.kv_read(ops.KvCache(None, None), i)
    with pytest.raises(ValueError, match="dimensions"):
        ops.kv_read(ops.KvCache(k, k), i)
    with pytest.raises(ValueError, match="dtype"):
        ops.kv_read(host, i, dtype=torch.int8)


def test_slots_of_page_numbers_that_no_cache_has():
    # 2^28 * 16 is 0 in 32 bits: a token of no page must not land in page 0
    big = 1 << 28
    table = torch.tensor([[big], [(1 << 31) - 1], [-1], [(1 << 27) - 1]], dtype=torch.int32)
    lengths = torch.full((4,), 3, dtype=torch.int32)
    got = fp8_layer.new_slots(table, lengths, 2, 16)
    assert got.dtype == torch.int32
    assert got.tolist() == [[-1, -1]] * 3 + [[(1 << 31) - 15, (1 << 31) - 14]]


@pytest.mark.parametrize("scale", [2.0 ** 127, -3e38])
def test_scales_that_no_product_with_them_is_finite(scale):
    refused(N.moeop_attend_paged, config(scale=scale), cache(), *attend_args(), text="scale")
