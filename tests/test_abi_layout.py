"""Structures that callers pass by address keep the layout that they had before
MXFP4 weights: a caller built on that header hands over as many bytes as the
library reads."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <stddef.h>
#include <stdio.h>
#include "soup.h"
/* the structures as they were with NF4 and bf16 weights alone */
typedef struct { int32_t kind; int64_t out_features, in_features; const uint8_t* codes; const float* absmax;
                 const uint16_t* w; } old_weight;
typedef struct { old_weight qkv, o, gate_up, down; const uint16_t *norm1, *norm2; } old_layer;
#define SAME(T, U, f) if (offsetof(T, f) != offsetof(U, f)) { printf(#T "." #f "\n"); bad = 1; }
int main(void) {
  int bad = 0;
  SAME(soup_weight, old_weight, out_features) SAME(soup_weight, old_weight, in_features)
  SAME(soup_weight, old_weight, codes) SAME(soup_weight, old_weight, absmax) SAME(soup_weight, old_weight, w)
  SAME(soup_layer_weights, old_layer, o) SAME(soup_layer_weights, old_layer, gate_up)
  SAME(soup_layer_weights, old_layer, down) SAME(soup_layer_weights, old_layer, norm1)
  SAME(soup_layer_weights, old_layer, norm2)
  if (sizeof(soup_weight) != sizeof(old_weight) || sizeof(soup_layer_weights) != sizeof(old_layer)) bad = 1;
  printf("%d %d %d %d %d\n", (int)sizeof(soup_weight), (int)sizeof(soup_layer_weights), (int)offsetof(soup_weight, codes),
         (int)offsetof(soup_weight, scales), (int)offsetof(soup_weight, w));
  return bad;
}
"""


@pytest.mark.parametrize("compiler", [["gcc", "-x", "c"], ["g++", "-x", "c++"]])
def test_weight_structures_keep_their_layout(compiler, tmp_path):
    exe = tmp_path / "layout"
    src = tmp_path / "layout.c"
    src.write_text(PROGRAM)
    subprocess.run([*compiler, "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    from layer_streamed_qlora_b200 import _lib as L
    assert [int(v) for v in r.stdout.split()] == [ctypes.sizeof(L.SoupWeight), ctypes.sizeof(L.LayerWeights),
                                                 L.SoupWeight.codes.offset, L.SoupWeight.absmax.offset,
                                                 L.SoupWeight.w.offset]


def test_a_weight_has_absmax_or_scales():
    from layer_streamed_qlora_b200 import _lib as L
    assert L.SoupWeight(L.SOUP_WEIGHT_MXFP4, 64, 96, 16, None, None, 32).scales == 32
    assert L.SoupWeight(L.SOUP_WEIGHT_NF4, 64, 64, 16, 48, None).absmax == 48
    with pytest.raises(ValueError, match="one field"):
        L.SoupWeight(L.SOUP_WEIGHT_MXFP4, 64, 96, 16, 48, None, 32)
