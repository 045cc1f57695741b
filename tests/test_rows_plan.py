"""Plans of prompt and tree attention follow the current device (CPU only, against the stand-in for the
CUDA runtime): workspaces by its SMs, and calls that fit them."""
from test_host_devices import RUNTIME, run_host

SMS = "static const int kSms[] = {152, 76, 40};\n"
MAIN = RUNTIME.replace("cudaDeviceAttr a, int) {", "cudaDeviceAttr a, int device) {").replace("? 152 : 0", "? kSms[device] : 0").replace(
    "static int g_device", SMS + "static int g_device", 1) + r"""
int main() {
  int fails = 0;
  for (int device : {0, 1, 2, 0})
    for (int units : {2, 16, 40, 64, 80})
      for (int n : {1, 20, 64}) {
        g_device = device;
        const bs_dims d = dims_for(BS_BF16, units, 8000, 8000);
        const bs_head_cfg c = cfg();
        const bs_kv k = cache();
        const size_t pw = bs_prefill_workspace_size(&d, 1000, n), tw = bs_tree_workspace_size(&d, n);
        const bs_drafts dr{P(21), P(22), 16 * 128, 1000, P(3), P(4), (const uint64_t *)P(5), n};
        std::printf("%d %d %d %zu %zu\n", kSms[device], units, n, pw, tw);
        auto prefill = [&](size_t bytes) {
          return bs_prefill_attn(&d, P(20), 8 * 128, 1000, &k, &c, P(2), P(3), n, P(33), nullptr, P(35), bytes, P(36), nullptr);
        };
        auto tree = [&](size_t bytes) {
          return bs_tree_decode_attn(&d, P(20), 8 * 128, &k, &c, P(27), P(28), &dr, P(33), nullptr, P(35), bytes, P(36), nullptr);
        };
        fails += prefill(pw) != BS_OK || tree(tw) != BS_OK;
        fails += (pw > 0 && prefill(pw - 1) != BS_ERR_CAPACITY) || (tw > 0 && tree(tw - 1) != BS_ERR_CAPACITY);
      }
  std::printf("fails %d\n", fails);
  return fails != 0;
}
"""


def test_plans_follow_the_device(tmp_path):
    r = run_host(tmp_path, MAIN)
    assert r.returncode == 0, r.stdout + r.stderr
    size = {}
    for line in r.stdout.splitlines()[:-1]:
        sms, units, n, prefill, tree = (int(x) for x in line.split())
        assert size.setdefault((sms, units, n), (prefill, tree)) == (prefill, tree)
    d = 128
    for sms in (152, 76, 40):
        for units, n, rows in ((16, 20, 80), (16, 64, 256)):      # a wave of CTAs shares these units' tiles
            assert size[sms, units, n][1] == sms * rows * (4 * d + 8) + 16 * units
        # two units' prompts of few rows over 4000 tiles: 167 pieces a unit, in eight waves at most
        assert size[sms, 2, 20][0] == 2 * min(167, 4 * sms) * 80 * (4 * d + 8) + 16 * 2
    # more units than CTAs: no wave that could share them (256 rows: whole units, no records)
    assert size[40, 64, 64][1] == 0 and size[40, 40, 64][1] > 0 and size[152, 64, 64][1] > 0
    assert size[76, 80, 64][1] == 0
