// Host helpers that the operators' launchers share with rssm_host.cu.
#pragma once

namespace rssm {

int num_sms();  // SMs a persistent grid is sized for; 0: no device

}  // namespace rssm
