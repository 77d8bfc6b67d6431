// kv_attention.cu - attention over the paged NVFP4 key/value cache: sizes of the
// workspace, and the kernels of the causal mask or none.
#include "kv_attention_launch.cuh"

namespace fp4q {
namespace {

template <int D, int NT>
int64_t decode_workspace(int sms, int64_t B, int64_t T, int group, int heads) {
  using S = DecodeShape<D, NT>;
  return 4LL * (2LL * sms * S::kCtas * S::kPart) + 8LL * decode_row_slots(B, T, group, S::kRows) * heads;
}

}  // namespace

void kv_attention_shape(int sms, int64_t B, int64_t T, int Hq, int heads, int D, int64_t keys, int64_t out[2]) {
  const int group = Hq / heads, nt = decode_tiles(B, T, group);
  out[0] = use_prefill(sms, B, T, Hq, heads, D, keys) ? 1 : 0;
  out[1] = out[0]     ? prefill_splits(sms, B, T, Hq, heads, D, keys, nullptr)
           : D == 128 ? (nt == 1 ? cluster_of<128, 1>(sms, B, T, group, heads, keys)
                                 : cluster_of<128, 2>(sms, B, T, group, heads, keys))
                      : (nt == 1 ? cluster_of<64, 1>(sms, B, T, group, heads, keys)
                                 : cluster_of<64, 2>(sms, B, T, group, heads, keys));
}

int64_t kv_attention_workspace(int sms, int64_t B, int64_t T, int Hq, int heads, int D, int64_t keys) {
  if (B == 0 || T == 0) return 0;
  int64_t shape[2];
  kv_attention_shape(sms, B, T, Hq, heads, D, keys, shape);
  if (shape[0]) return shape[1] > 1 ? shape[1] * T * Hq * (D + 2) * 4 : 0;
  if (shape[1]) return 0;
  const int group = Hq / heads;
  if (D == 128)
    return decode_tiles(B, T, group) == 1 ? decode_workspace<128, 1>(sms, B, T, group, heads)
                                          : decode_workspace<128, 2>(sms, B, T, group, heads);
  return decode_tiles(B, T, group) == 1 ? decode_workspace<64, 1>(sms, B, T, group, heads)
                                        : decode_workspace<64, 2>(sms, B, T, group, heads);
}

// The decode kernel's size grows with B and T.  The other's is splits * T * Hq * (D + 2)
// floats, where the splits are those that prefill_splits may choose: items * splits <= 4
// SMs, and the items are T * Hq / 256 or more.
int64_t kv_attention_workspace_bound(int sms, int64_t B, int64_t T, int Hq, int heads, int D, int64_t keys) {
  if (B == 0 || T == 0) return 0;
  const int group = Hq / heads;
  const int64_t decode = D == 128 ? std::max(decode_workspace<128, 1>(sms, B, T, group, heads),
                                             decode_workspace<128, 2>(sms, B, T, group, heads))
                                  : std::max(decode_workspace<64, 1>(sms, B, T, group, heads),
                                             decode_workspace<64, 2>(sms, B, T, group, heads));
  const int64_t splits = std::min<int64_t>(kPreMostSplits, (keys + kPreKeys - 1) / kPreKeys);
  const int64_t rows = splits > 1 ? std::min<int64_t>(splits * T * Hq, 4LL * sms * kPreRows) : 0;
  return std::max(decode, rows * (D + 2) * 4);
}

cudaError_t launch_kv_attention(int dtype, const KvAttentionParams& p, int pdl,
                                cudaStream_t stream) {
  return launch_attention<kPlain, kPlain>(dtype, p, pdl, stream);
}

}  // namespace fp4q
