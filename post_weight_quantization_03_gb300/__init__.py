"""GB300-native GPTQ per-layer quantization, and 8-bit serving of the quantized layers: a C-ABI CUDA library plus a thin binding."""
